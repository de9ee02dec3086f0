// kda_block_norm.cu -- the norms around a block, one pass over each row:
//     n  = y / rms(y) * w_post      per group of channels (a head, or the row)
//     u  = n * act(gate)            act = sigmoid or silu
//     x' = x + res_scale * u
//     h  = x' / rms(x') * w_pre
// and its backward.  All of it is bound by the bytes of the rows: each tensor
// is read or written once, the row stays in registers between the two norms,
// statistics and sums are fp32.
#include "kda_block_norm.h"

#include <cuda_bf16.h>

namespace kda {
namespace {

constexpr int V = 8;             // channels per vector: 16 bytes of bf16
constexpr int MAX_THREADS = 512;
constexpr int MAX_PARTS = 304;   // two CTAs on each of 152 SMs
constexpr int MAX_ROWS = 4;      // rows that short-row blocks take at once

__device__ __forceinline__ void load(const float* p, float (&v)[V]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[V]) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store(float* p, const float (&v)[V]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[V]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float sigmoid(float t) { return 1.0f / (1.0f + expf(-t)); }

// Sums of M values over the `width` consecutive lanes (a power of two) of the
// calling thread.
template <int M>
__device__ __forceinline__ void lane_sum(float (&s)[M], int width) {
    for (int m = width / 2; m > 0; m >>= 1) {
#pragma unroll
        for (int i = 0; i < M; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], m);
    }
}

// Sums over the warps of a row (all threads of the block call it; threadIdx.y
// is the row).  `turn` alternates between two halves of the buffer, so that
// one barrier per sum is enough.
template <int M>
__device__ __forceinline__ void row_sum(float (&s)[M], float* buf, int warps, int turn) {
    lane_sum(s, 32);
    if (warps == 1) return;
    float* b = buf + (turn * blockDim.y + threadIdx.y) * (32 * 3);
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < M; ++i) b[w * 3 + i] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) s[i] = 0.0f;
    for (int j = 0; j < warps; ++j) {
#pragma unroll
        for (int i = 0; i < M; ++i) s[i] += b[j * 3 + i];
    }
}

// Block shape: threadIdx.x over the vectors of a row's tile (whole warps), VPT
// vectors per thread, threadIdx.y over rows; blockIdx.y over the tiles, of
// which there is only one where a sum runs over the whole row.
template <typename T, int VPT>
__global__ void __launch_bounds__(MAX_THREADS) block_norm_kernel(BlockNorm p, int tile) {
    __shared__ float buf[2 * MAX_ROWS * 32 * 3];
    const int warps = blockDim.x >> 5;
    const int vec0 = blockIdx.y * tile / V + threadIdx.x;
    const int vecs = min(p.D, ((int)blockIdx.y + 1) * tile) / V;
    const bool whole = p.group == p.D;
    const int lanes = whole ? 32 : p.group / V;
    const T* y = static_cast<const T*>(p.y);
    const T* gate = static_cast<const T*>(p.gate);
    const T* x = static_cast<const T*>(p.x);
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < p.rows; r0 += step) {
        const int64_t row = r0 + threadIdx.y;
        const bool live = row < p.rows;
        float u[VPT][V], xs[VPT][V], gt[VPT][V];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = vec0 + i * blockDim.x;
            const size_t at = (size_t)row * p.D + (size_t)vec * V;
            const bool in = live && vec < vecs;
#pragma unroll
            for (int e = 0; e < V; ++e) { u[i][e] = 0.f; xs[i][e] = 0.f; gt[i][e] = 0.f; }
            if (in) {
                load(y + at, u[i]);
                if (gate) load(gate + at, gt[i]);
                if (x) load(x + at, xs[i]);
            }
        }
        float ss[VPT][1];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            ss[i][0] = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) ss[i][0] += u[i][e] * u[i][e];
        }
        if (whole) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < VPT; ++i) s[0] += ss[i][0];
            row_sum(s, buf, warps, 0);
#pragma unroll
            for (int i = 0; i < VPT; ++i) ss[i][0] = s[0];
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) lane_sum(ss[i], lanes);
        }
        float s2[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = vec0 + i * blockDim.x;
            if (!live || vec >= vecs) continue;
            const float r = rsqrtf(ss[i][0] / (float)p.group + p.eps);
            float w[V];
            load(p.w_post + (vec * V) % p.group, w);
#pragma unroll
            for (int e = 0; e < V; ++e) u[i][e] = u[i][e] * r * w[e];
            if (gate) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float a = sigmoid(gt[i][e]);
                    u[i][e] *= p.silu ? gt[i][e] * a : a;
                }
            }
            if (p.res_scale) {
                load(p.res_scale + vec * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) u[i][e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                u[i][e] += xs[i][e];
                s2[0] += u[i][e] * u[i][e];
            }
            store(static_cast<T*>(p.x_out) + (size_t)row * p.D + (size_t)vec * V, u[i]);
        }
        if (p.w_pre) {
            row_sum(s2, buf, warps, 1);
            const float r = rsqrtf(s2[0] / (float)p.D + p.eps);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = vec0 + i * blockDim.x;
                if (!live || vec >= vecs) continue;
                float w[V];
                load(p.w_pre + vec * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) u[i][e] = u[i][e] * r * w[e];
                store(static_cast<T*>(p.h) + (size_t)row * p.D + (size_t)vec * V, u[i]);
            }
        }
        if (warps > 1 && (whole != (p.w_pre != nullptr))) __syncthreads();   // one sum a row: the
        // next row writes the half that this row still reads
    }
}

// Per row, with r = 1 / rms and the upstream gradients dX of x' and dh of h:
//     total  = dX + r (dh w_pre) - x' r^3 mean(dh w_pre x')        (= dx)
//     dy     = r dn - y r^3 mean(dn y),   dn = total res_scale act(gate) w_post
//     dgate  = total res_scale n act'(gate)
// and over the rows: dw_pre += dh x' r, dres_scale += total u,
// dw_post += total res_scale act(gate) y r.  The rows of a CTA add to
// registers; each CTA leaves its sums apart and a second kernel adds them in
// order, so that a repeated call gives the same bits.
template <typename T, int VPT>
__global__ void __launch_bounds__(MAX_THREADS) block_norm_backward_kernel(BlockNorm p, int tile) {
    __shared__ float buf[2 * MAX_ROWS * 32 * 3];
    const int warps = blockDim.x >> 5;
    const int vec0 = blockIdx.y * tile / V + threadIdx.x;
    const int vecs = min(p.D, ((int)blockIdx.y + 1) * tile) / V;
    const bool whole = p.group == p.D;
    const int lanes = whole ? 32 : p.group / V;
    const T* y = static_cast<const T*>(p.y);
    const T* gate = static_cast<const T*>(p.gate);
    const T* x = static_cast<const T*>(p.x);
    const T* dxo = static_cast<const T*>(p.dx_out);
    const T* dh = static_cast<const T*>(p.dh);
    float a_post[VPT][V], a_res[VPT][V], a_pre[VPT][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) a_post[i][e] = a_res[i][e] = a_pre[i][e] = 0.f;

    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < p.rows; r0 += step) {
        const int64_t row = r0 + threadIdx.y;
        const bool live = row < p.rows;
        float yv[VPT][V], gt[VPT][V], tot[VPT][V], ry[VPT];
        float s[3] = {0.f, 0.f, 0.f};   // x'^2, dh w_pre x', y^2
        float xv[VPT][V], dn[VPT][V];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = vec0 + i * blockDim.x;
            const size_t at = (size_t)row * p.D + (size_t)vec * V;
            const bool in = live && vec < vecs;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                yv[i][e] = gt[i][e] = tot[i][e] = xv[i][e] = dn[i][e] = 0.f;
            }
            if (in) {
                load(y + at, yv[i]);
                if (gate) load(gate + at, gt[i]);
                if (dxo) load(dxo + at, tot[i]);
                if (p.w_pre) {
                    load(x + at, xv[i]);
                    load(dh + at, dn[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = vec0 + i * blockDim.x;
            float w[V], yy[1] = {0.f};
            if (p.w_pre && vec < vecs) {
                load(p.w_pre + vec * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s[0] += xv[i][e] * xv[i][e];
                    s[1] += dn[i][e] * w[e] * xv[i][e];
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) yy[0] += yv[i][e] * yv[i][e];
            if (whole) {
                s[2] += yy[0];
            } else {
                lane_sum(yy, lanes);
                ry[i] = rsqrtf(yy[0] / (float)p.group + p.eps);
            }
        }
        const bool sums = whole || p.w_pre;
        if (sums) row_sum(s, buf, warps, 0);
        if (whole) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) ry[i] = rsqrtf(s[2] / (float)p.D + p.eps);
        }
        float s2[1] = {0.f};
        float cy[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = vec0 + i * blockDim.x;
            const bool in = live && vec < vecs;
            const size_t at = (size_t)row * p.D + (size_t)vec * V;
            float w[V];
            if (in && p.w_pre) {
                const float r = rsqrtf(s[0] / (float)p.D + p.eps);
                const float c = s[1] / (float)p.D * r * r * r;
                load(p.w_pre + vec * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    a_pre[i][e] += dn[i][e] * xv[i][e] * r;
                    tot[i][e] += r * dn[i][e] * w[e] - xv[i][e] * c;
                }
            }
            if (in && p.dx) store(static_cast<T*>(p.dx) + at, tot[i]);
            float part[1] = {0.f};
            if (in) {
                float act[V], slope[V];
#pragma unroll
                for (int e = 0; e < V; ++e) { act[e] = 1.f; slope[e] = 0.f; }
                if (gate) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float t = gt[i][e], a = sigmoid(t);
                        act[e] = p.silu ? t * a : a;
                        slope[e] = p.silu ? a * (1.f + t * (1.f - a)) : a * (1.f - a);
                    }
                }
                float rs[V];
#pragma unroll
                for (int e = 0; e < V; ++e) rs[e] = 1.f;
                if (p.res_scale) load(p.res_scale + vec * V, rs);
                load(p.w_post + (vec * V) % p.group, w);
                float dg[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float yn = yv[i][e] * ry[i], n = yn * w[e];
                    a_res[i][e] += tot[i][e] * n * act[e];
                    const float du = tot[i][e] * rs[e];
                    dg[e] = du * n * slope[e];
                    a_post[i][e] += du * act[e] * yn;
                    tot[i][e] = du * act[e] * w[e];   // dn from here on
                    part[0] += tot[i][e] * yv[i][e];
                }
                if (gate) store(static_cast<T*>(p.dgate) + at, dg);
            }
            if (whole) {
                s2[0] += part[0];
            } else {
                lane_sum(part, lanes);
                cy[i] = part[0] / (float)p.group;
            }
        }
        if (whole) {
            row_sum(s2, buf, warps, 1);
#pragma unroll
            for (int i = 0; i < VPT; ++i) cy[i] = s2[0] / (float)p.D;
        } else if (sums && warps > 1) {
            __syncthreads();   // the next row writes the sums this row has read
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = vec0 + i * blockDim.x;
            if (!live || vec >= vecs) continue;
            const float r = ry[i], c = cy[i] * r * r * r;
#pragma unroll
            for (int e = 0; e < V; ++e) tot[i][e] = r * tot[i][e] - yv[i][e] * c;
            store(static_cast<T*>(p.dy) + (size_t)row * p.D + (size_t)vec * V, tot[i]);
        }
    }

    // sums of this block's rows: threadIdx.y groups in order, then one part per CTA
    extern __shared__ float4 dyn4[];
    float* dyn = reinterpret_cast<float*>(dyn4);   // [3][D] when blockDim.y > 1
    float* mine = p.partial + (size_t)blockIdx.x * 3 * p.D;
    float* sum = blockDim.y > 1 ? dyn : mine;
    for (unsigned k = 0; k < blockDim.y; ++k) {
        if (threadIdx.y == k) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = vec0 + i * blockDim.x;
                if (vec >= vecs) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int c = vec * V + e;
                    sum[c] = (k ? sum[c] : 0.f) + a_post[i][e];
                    sum[p.D + c] = (k ? sum[p.D + c] : 0.f) + a_res[i][e];
                    sum[2 * p.D + c] = (k ? sum[2 * p.D + c] : 0.f) + a_pre[i][e];
                }
            }
        }
        if (blockDim.y > 1) __syncthreads();
    }
    if (blockDim.y > 1) {
        for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < 3 * p.D;
             c += blockDim.x * blockDim.y)
            mine[c] = dyn[c];
    }
}

// One CTA per 32 columns of one of the three sums: parts in order within each
// of 8 rows of threads, then the rows in order.  dw_post of a head also adds
// the heads.
__global__ void block_norm_sums_kernel(BlockNorm p, int parts) {
    __shared__ float buf[8][33];
    const int which = blockIdx.y;
    float* dst = which == 0 ? p.dw_post : which == 1 ? p.dres_scale : p.dw_pre;
    const int width = which == 0 ? p.group : p.D;
    if (!dst) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    if (blockIdx.x * 32 >= width) return;
    float s = 0.f;
    if (c < width) {
        for (int k = threadIdx.y; k < parts; k += 8) {
            const float* part = p.partial + ((size_t)k * 3 + which) * p.D;
            for (int at = c; at < p.D; at += width) s += part[at];
        }
    }
    buf[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < width) {
        for (int k = 1; k < 8; ++k) s += buf[k][threadIdx.x];
        dst[c] = s;
    }
}

struct Shape {
    dim3 block;
    int vpt;
    int tile;    // columns per block
    int tiles;
};

// Up to 512 threads on a row; short rows share a block of 128 threads.  Where
// no sum runs over the row (heads, no pre norm) a wide one is cut into tiles of
// 2048 columns, blocks of their own.
Shape shape_of(int32_t D, bool coupled) {
    Shape s;
    s.tile = coupled || D <= 2048 ? D : 2048;
    s.tiles = (D + s.tile - 1) / s.tile;
    const int vecs = s.tile / V;
    s.vpt = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
    const int tx = ((vecs + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    s.block = dim3(tx, tx >= 128 ? 1 : 128 / tx);
    return s;
}

bool coupled(const BlockNorm& p) { return p.group == p.D || p.w_pre; }

template <typename T>
cudaError_t forward(const BlockNorm& p, cudaStream_t stream) {
    const Shape s = shape_of(p.D, coupled(p));
    const int64_t rows = (p.rows + s.block.y - 1) / s.block.y, most = 152 * 16 / s.tiles;
    const dim3 grid((unsigned)(rows < most ? rows : most), s.tiles);
    switch (s.vpt) {
        case 1: block_norm_kernel<T, 1><<<grid, s.block, 0, stream>>>(p, s.tile); break;
        case 2: block_norm_kernel<T, 2><<<grid, s.block, 0, stream>>>(p, s.tile); break;
        default: block_norm_kernel<T, 4><<<grid, s.block, 0, stream>>>(p, s.tile); break;
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const BlockNorm& p, cudaStream_t stream) {
    const Shape s = shape_of(p.D, coupled(p));
    const int parts = block_norm_parts(p.rows, p.D);
    const dim3 grid(parts, s.tiles);
    // rows that share a block add their sums in shared memory (one tile then)
    const size_t smem = s.block.y > 1 ? (size_t)3 * p.D * sizeof(float) : 0;
    switch (s.vpt) {
        case 1:
            block_norm_backward_kernel<T, 1><<<grid, s.block, smem, stream>>>(p, s.tile);
            break;
        case 2:
            block_norm_backward_kernel<T, 2><<<grid, s.block, smem, stream>>>(p, s.tile);
            break;
        default:
            block_norm_backward_kernel<T, 4><<<grid, s.block, smem, stream>>>(p, s.tile);
            break;
    }
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    block_norm_sums_kernel<<<dim3((p.D + 31) / 32, 3), dim3(32, 8), 0, stream>>>(p, parts);
    return cudaGetLastError();
}

}  // namespace

int block_norm_parts(int64_t rows, int32_t D) {
    const int64_t y = shape_of(D, true).block.y, blocks = (rows + y - 1) / y;
    return (int)(blocks < MAX_PARTS ? (blocks < 1 ? 1 : blocks) : MAX_PARTS);
}

cudaError_t launch_block_norm(const BlockNorm& p, int dtype, cudaStream_t stream) {
    return dtype == 0 ? forward<float>(p, stream) : forward<__nv_bfloat16>(p, stream);
}

cudaError_t launch_block_norm_backward(const BlockNorm& p, int dtype, cudaStream_t stream) {
    return dtype == 0 ? backward<float>(p, stream) : backward<__nv_bfloat16>(p, stream);
}

}  // namespace kda
