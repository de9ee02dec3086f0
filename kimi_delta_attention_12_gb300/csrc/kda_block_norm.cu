// kda_block_norm.cu -- the norms around a block, one pass over each row:
//     n  = y / rms(y) * w_post      per group of channels (a head, or the row)
//     u  = n * act(gate)            act = sigmoid or silu
//     x' = x + res_scale * u
//     h  = x' / rms(x') * w_pre
// and its backward.  All of it is bound by the bytes of the rows: each tensor
// is read or written once, the row stays in registers between the two norms,
// statistics and sums are fp32.  What that takes is bytes in flight: a thread
// has the loads of its next row (or of four vectors, where rows do not matter)
// under way while it works.  65,536 rows of 96 heads of 128, gated, bf16: 785 us,
// 6.15 TB/s (0.91 of a plain copy's rate; row by row they took 1,408).  One row of
// 4,096: 5 us on the device, two sums over a block after one trip to memory.
#include "kda_block_norm.h"

#include <cuda_bf16.h>
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "kda_follow.cuh"
#include "kda_packed.cuh"

namespace kda {
namespace {

constexpr int V = 8;             // channels per vector: 16 bytes of bf16
constexpr int MAX_THREADS = 512;
constexpr int MAX_ROWS = 4;      // rows that short-row blocks take at once
constexpr int TILE = 2048;       // columns per block where rows do not couple them
constexpr int SUMS = 2 * MAX_ROWS * 32 * 3;   // row_sum's buffer

// A vector as it was loaded.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    float4 a, b;
};
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
};

__device__ __forceinline__ void fetch(const float* p, Raw<float>& r) {
    r.a = *reinterpret_cast<const float4*>(p);
    r.b = *reinterpret_cast<const float4*>(p + 4);
}
__device__ __forceinline__ void fetch(const __nv_bfloat16* p, Raw<__nv_bfloat16>& r) {
    r.a = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void clear(Raw<float>& r) {
    r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f);
}
__device__ __forceinline__ void clear(Raw<__nv_bfloat16>& r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void expand(const Raw<float>& r, float (&v)[V]) {
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
__device__ __forceinline__ void expand(const Raw<__nv_bfloat16>& r, float (&v)[V]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load(const float* p, float (&v)[V]) {
    Raw<float> r;
    fetch(p, r);
    expand(r, v);
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

// 1 / (1 + e^-t).  fp32: a few units in the last place.  bf16 rows: from the
// approximate 2^x and reciprocal, relative error near 2^-22 (1 + |t|), which
// the rounding of the gate itself (2^-8) hides, in 4 instructions instead of 14:
// with the full expf 65,536 rows of 96 heads took 885 us where they take 780.
template <typename T>
__device__ __forceinline__ float sigmoid(float t);
template <>
__device__ __forceinline__ float sigmoid<float>(float t) {
    return __fdividef(1.0f, 1.0f + expf(-t));
}
template <>
__device__ __forceinline__ float sigmoid<__nv_bfloat16>(float t) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// A vector as four pairs.
__device__ __forceinline__ void expand2(const Raw<float>& r, uint64_t (&v)[V / 2]) {
    v[0] = two(r.a.x, r.a.y); v[1] = two(r.a.z, r.a.w);
    v[2] = two(r.b.x, r.b.y); v[3] = two(r.b.z, r.b.w);
}
__device__ __forceinline__ void expand2(const Raw<__nv_bfloat16>& r, uint64_t (&v)[V / 2]) {
    v[0] = two(low(r.a.x), high(r.a.x)); v[1] = two(low(r.a.y), high(r.a.y));
    v[2] = two(low(r.a.z), high(r.a.z)); v[3] = two(low(r.a.w), high(r.a.w));
}
__device__ __forceinline__ void load2(const float* p, uint64_t (&v)[V / 2]) {
    Raw<float> r;
    fetch(p, r);
    expand2(r, v);
}
__device__ __forceinline__ void store2(float* p, const uint64_t (&v)[V / 2]) {
    float f[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) apart(v[i], f[2 * i], f[2 * i + 1]);
    store(p, f);
}
__device__ __forceinline__ void store2(__nv_bfloat16* p, const uint64_t (&v)[V / 2]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack(v[0]), pack(v[1]), pack(v[2]), pack(v[3]));
}

// Sums of M values over the `width` consecutive lanes (a power of two) of the
// calling thread.
template <int M>
__device__ __forceinline__ void lane_sum(float (&s)[M], int width) {
    for (int m = width / 2; m > 0; m >>= 1) {
#pragma unroll
        for (int i = 0; i < M; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], m);
    }
}

// The threads of one row wait for one another (threadIdx.y is the row; a block
// has two rows of several warps at most).
__device__ __forceinline__ void row_wait() {
    if (threadIdx.y == 0) {
        asm volatile("bar.sync 1, %0;" ::"r"(blockDim.x) : "memory");
    } else {
        asm volatile("bar.sync 2, %0;" ::"r"(blockDim.x) : "memory");
    }
}

// Sums over the warps of a row (all threads of the row call it).  `turn`
// alternates between two halves of the buffer, so that one barrier per sum is
// enough.
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
    row_wait();
    // every warp adds the (up to 16) warps' sums itself, in each half or quarter of its lanes
    const int lane = threadIdx.x & (warps <= 8 ? 7 : 15);
#pragma unroll
    for (int i = 0; i < M; ++i) s[i] = lane < warps ? b[lane * 3 + i] : 0.0f;
    if (warps <= 8) {
        lane_sum(s, 8);
    } else {
        lane_sum(s, 16);
    }
}

// n act(gate) res_scale of one vector; y replaced by it.
template <typename T>
__device__ __forceinline__ void branch(float (&u)[V], const float (&g)[V], float r,
                                       const float* w_post, const float* res, bool gate,
                                       int silu) {
    float w[V];
    load(w_post, w);
#pragma unroll
    for (int e = 0; e < V; ++e) u[e] = u[e] * r * w[e];
    if (gate) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float a = sigmoid<T>(g[e]);
            u[e] *= silu ? g[e] * a : a;
        }
    }
    if (res) {
        load(res, w);
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] *= w[e];
    }
}

// ------------------------------------------------------------ forward, heads
// No sum runs over a row: the tensors are streams of vectors, a group's lanes
// side by side.  Four vectors a thread, all loads first.
template <typename T>
__global__ void __launch_bounds__(256) block_norm_heads_kernel(BlockNorm p, int64_t vecs) {
    constexpr int U = 4;
    const int lanes = p.group / V;
    const int64_t first = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
    const T* y = static_cast<const T*>(p.y);
    const T* gate = static_cast<const T*>(p.gate);
    const T* x = static_cast<const T*>(p.x);
    Raw<T> ry[U], rg[U], rx[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t vec = first + 256 * i;
        clear(ry[i]);
        clear(rg[i]);
        clear(rx[i]);
        if (vec < vecs) {
            fetch(y + vec * V, ry[i]);
            if (gate) fetch(gate + vec * V, rg[i]);
            if (x) fetch(x + vec * V, rx[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t vec = first + 256 * i;
        float u[V], g[V], xs[V], s[1] = {0.f};
        expand(ry[i], u);
        expand(rg[i], g);
        expand(rx[i], xs);
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += u[e] * u[e];
        lane_sum(s, lanes);
        if (vec >= vecs) continue;
        const float* res =
            p.res_scale ? p.res_scale + (vec % (p.D / V)) * V : nullptr;
        branch<T>(u, g, rsqrtf(s[0] / (float)p.group + p.eps),
               p.w_post + (int)(vec & (lanes - 1)) * V, res, gate != nullptr, p.silu);
        if (x) {
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] += xs[e];
        }
        store(static_cast<T*>(p.x_out) + vec * V, u);
    }
}

// ------------------------------------------------------------- forward, rows
// Block shape: threadIdx.x over the vectors of a row (whole warps), VPT
// vectors per thread, threadIdx.y over rows.
template <typename T, int VPT>
__global__ void __launch_bounds__(MAX_THREADS) block_norm_kernel(BlockNorm p) {
    __shared__ float buf[SUMS];
    const int warps = blockDim.x >> 5, vecs = p.D / V;
    const bool whole = p.group == p.D;
    const int lanes = whole ? 32 : p.group / V;
    const T* y = static_cast<const T*>(p.y);
    const T* gate = static_cast<const T*>(p.gate);
    const T* x = static_cast<const T*>(p.x);
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    Raw<T> ry[VPT], rg[VPT], rx[VPT];
    auto fetch_row = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = threadIdx.x + i * blockDim.x;
            clear(ry[i]);
            clear(rg[i]);
            clear(rx[i]);
            if (row < p.rows && vec < vecs) {
                const size_t at = (size_t)row * p.D + (size_t)vec * V;
                fetch(y + at, ry[i]);
                if (gate) fetch(gate + at, rg[i]);
                if (x) fetch(x + at, rx[i]);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    fetch_row(row);
    for (; row < p.rows; row += step) {
        float u[VPT][V];
        Raw<T> cg[VPT], cx[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            expand(ry[i], u[i]);
            cg[i] = rg[i];
            cx[i] = rx[i];
        }
        fetch_row(row + step);
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
            const int vec = threadIdx.x + i * blockDim.x;
            if (vec >= vecs) continue;
            float g[V], xs[V];
            expand(cg[i], g);
            expand(cx[i], xs);
            branch<T>(u[i], g, rsqrtf(ss[i][0] / (float)p.group + p.eps),
                   p.w_post + (whole ? vec : vec & (lanes - 1)) * V,
                   p.res_scale ? p.res_scale + vec * V : nullptr, gate != nullptr, p.silu);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (x) u[i][e] += xs[e];
                s2[0] += u[i][e] * u[i][e];
            }
            store(static_cast<T*>(p.x_out) + (size_t)row * p.D + (size_t)vec * V, u[i]);
        }
        if (p.w_pre) {
            row_sum(s2, buf, warps, 1);
            const float r = rsqrtf(s2[0] / (float)p.D + p.eps);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = threadIdx.x + i * blockDim.x;
                if (vec >= vecs) continue;
                float w[V];
                load(p.w_pre + vec * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) u[i][e] = u[i][e] * r * w[e];
                store(static_cast<T*>(p.h) + (size_t)row * p.D + (size_t)vec * V, u[i]);
            }
        }
        if (warps > 1 && (whole != (p.w_pre != nullptr))) row_wait();   // one sum a row: the
        // next row writes the half that this row still reads
    }
}

// ------------------------------------------------------------------ backward
// Per row, with r = 1 / rms and the upstream gradients dX of x' and dh of h:
//     total  = dX + r (dh w_pre) - x' r^3 mean(dh w_pre x')        (= dx)
//     dy     = r dn - y r^3 mean(dn y),   dn = total res_scale act(gate) w_post
//     dgate  = total res_scale n act'(gate)
// and over the rows: dw_pre += dh x' r, dres_scale += total u,
// dw_post += total res_scale act(gate) y r.  The rows of a CTA add to
// registers; each CTA leaves its sums apart and a second kernel adds them in
// order, so that a repeated call gives the same bits.  blockIdx.y is the tile of
// columns, of which there is one where a sum runs over the row.
//
// RING: rows arrive in shared memory by asynchronous copies, `stages` of them
// under way or at work; a thread copies what it reads itself, so that its own
// wait is enough.  The registers that rows in flight would take go to the
// sums.  Rows too wide for that (stages = 0) are read into registers.
// FULL: a row's threads cover the columns exactly, so that nothing needs a guard.
// KEEP: every part is there (the norm over the row, both upstream gradients, dx), and
// the three weights are in shared memory too, for the block's rows: no branches for absent
// parts, and no row waits for weights that L1, beside the rings, is too small for.  Without
// and with it, sigmoid gate, 4,096 rows (8,192 below 2,048 columns), us, bf16: 256 columns 30,
// 30; 1,000 46, 40; 2,048 44, 37; 2,304 66, 46; 4,096 84, 60; 5,120 117, 78; 7,168 150, 100
// (4.7 TB/s, 69 % of a plain copy's); 8,192, for which it has no room, 166.  fp32: 1,000 94,
// 66; 2,304 100, 71; 4,096 161, 111.  What is left is the chain of a row: two sums over it,
// each a barrier, with 16 warps at most on an SM (128 registers a thread); the instructions
// alone would take 20 us at 4,096 columns.  64 registers and twice the warps spill.
enum { Y = 0, GATE = 1, DXO = 2, X = 3, DH = 4, TENSORS = 5 };

__device__ __forceinline__ void copy16(void* smem, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(smem)),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_done(int behind) {   // all but the last `behind` rows'
    if (behind >= 2) {
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    } else if (behind == 1) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
}

enum { NO_GATE = 0, SIGMOID = 1, SILU = 2 };

template <typename T, int VPT, int ACT, bool RING, bool FULL, bool KEEP = false>
__global__ void __launch_bounds__(MAX_THREADS)
block_norm_backward_kernel(BlockNorm p, int tile, int stages) {
    __shared__ float buf[SUMS];
    const int width = blockDim.x, rows = blockDim.y, D = p.D, cols = KEEP ? D : tile;
    const int depth = stages, warps = width >> 5;
    const int vec0 = KEEP ? (int)threadIdx.x : (int)(blockIdx.y * cols / V + threadIdx.x);
    const int vecs = KEEP ? D / V : min(D, ((int)blockIdx.y + 1) * cols) / V;
    const bool whole = KEEP || p.group == D, pre = KEEP || p.w_pre, pass_on = KEEP || p.dx;
    const int lanes = whole ? 32 : p.group / V;
    const T* src[TENSORS] = {static_cast<const T*>(p.y), static_cast<const T*>(p.gate),
                             static_cast<const T*>(p.dx_out),
                             static_cast<const T*>(pre ? p.x : nullptr),
                             static_cast<const T*>(pre ? p.dh : nullptr)};
    auto has = [&](int t) { return t == GATE ? ACT != NO_GATE : KEEP || src[t]; };
    extern __shared__ float4 dyn4[];
    uint64_t a_post[VPT][V / 2], a_res[VPT][V / 2], a_pre[VPT][V / 2];   // pairs
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < V / 2; ++e) a_post[i][e] = a_res[i][e] = a_pre[i][e] = 0;

    const int64_t step = (int64_t)gridDim.x * rows;
    int64_t row = (int64_t)blockIdx.x * rows + threadIdx.y;
    const int all = width * rows, flat = threadIdx.y * width + threadIdx.x;
    Raw<T>* ring = reinterpret_cast<Raw<T>*>(dyn4);   // [depth][TENSORS][VPT][all]
    float* kept = reinterpret_cast<float*>(ring + depth * TENSORS * VPT * all);   // [3][tile]
    if (KEEP) {
        for (int c = flat; c < cols; c += all) {
            kept[c] = p.w_post[c];
            kept[cols + c] = p.res_scale ? p.res_scale[c] : 1.0f;
            kept[2 * cols + c] = p.w_pre[c];
        }
        __syncthreads();
    }
    const float* w_post = KEEP ? kept : p.w_post;
    const float* res_scale = KEEP ? kept + cols : p.res_scale;
    const float* w_pre = KEEP ? kept + 2 * cols : p.w_pre;
    auto slot = [&](int stage, int k, int i) {
        return ring + ((stage * TENSORS + k) * VPT + i) * all + flat;
    };
    auto copy_row = [&](int64_t r, int stage) {
        if (r < p.rows) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = vec0 + i * width;
                if (!FULL && vec >= vecs) continue;
                const size_t at = (size_t)r * D + (size_t)vec * V;
#pragma unroll
                for (int k = 0; k < TENSORS; ++k) {
                    if (!has(k)) continue;
#pragma unroll
                    for (int q = 0; q < (int)sizeof(Raw<T>) / 16; ++q)
                        copy16(reinterpret_cast<uint4*>(slot(stage, k, i)) + q,
                               reinterpret_cast<const uint4*>(src[k] + at) + q);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");   // a group a row, empty or not
    };
    if (RING) {
        for (int k = 0; k + 1 < depth; ++k) copy_row(row + k * step, k);
    }
    int stage = 0;
    const float inv_row = 1.0f / (float)D, inv_group = 1.0f / (float)p.group;
    for (; row < p.rows; row += step) {
        Raw<T> held[RING ? 1 : TENSORS][RING ? 1 : VPT];
        if (RING) {
            // the stage that the row before has left takes the next row to come
            const int free = stage == 0 ? depth - 1 : stage - 1;
            copy_row(row + (depth - 1) * step, free);
            copies_done(depth - 1);
        } else {
#pragma unroll
            for (int k = 0; k < (RING ? 0 : TENSORS); ++k)
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int vec = vec0 + i * width;
                    clear(held[k][i]);
                    if (has(k) && vec < vecs)
                        fetch(src[k] + (size_t)row * D + (size_t)vec * V, held[k][i]);
                }
        }
        auto get = [&](int k, int i, uint64_t (&v)[V / 2]) {
            const bool in = FULL || vec0 + i * width < vecs;
            if (RING) {
                Raw<T> r;
                if (!FULL) clear(r);
                if (in) r = *slot(stage, k, i);
                expand2(r, v);
            } else {
                expand2(held[RING ? 0 : k][RING ? 0 : i], v);
            }
        };
        float s[3] = {0.f, 0.f, 0.f};   // x'^2, dh w_pre x', y^2
        float rr[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = vec0 + i * width;
            uint64_t a[V / 2], q0 = 0, q1 = 0, q2 = 0;
            if (pre && (FULL || vec < vecs)) {
                uint64_t w[V / 2], h[V / 2];
                get(X, i, a);
                get(DH, i, h);
                load2(w_pre + vec * V, w);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    q0 = fma2(a[e], a[e], q0);
                    q1 = fma2(mul2(h[e], w[e]), a[e], q1);
                }
            }
            get(Y, i, a);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) q2 = fma2(a[e], a[e], q2);
            s[0] += sum2(q0);
            s[1] += sum2(q1);
            if (whole) {
                s[2] += sum2(q2);
            } else {
                float yy[1] = {sum2(q2)};
                lane_sum(yy, lanes);
                rr[i] = rsqrtf(yy[0] * inv_group + p.eps);
            }
        }
        const bool sums = whole || pre;
        if (sums) row_sum(s, buf, warps, 0);
        if (whole) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) rr[i] = rsqrtf(s[2] * inv_group + p.eps);
        }
        const float rx = rsqrtf(s[0] * inv_row + p.eps);
        const uint64_t rx2 = two(rx, rx);
        const float cx = -s[1] * inv_row * rx * rx * rx;
        const uint64_t cx2 = two(cx, cx);
        float s2[1] = {0.f};
        uint64_t tot[VPT][V / 2];
        float cc[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = vec0 + i * width;
            const bool in = FULL || vec < vecs;
            const size_t at = (size_t)row * D + (size_t)vec * V;
            uint64_t w[V / 2], part = 0;
            if (KEEP) asm volatile("" ::: "memory");   // (loads ahead of their turn would spill)
            if (has(DXO)) {
                get(DXO, i, tot[i]);
            } else {
#pragma unroll
                for (int e = 0; e < V / 2; ++e) tot[i][e] = 0;
            }
            if (in && pre) {
                uint64_t a[V / 2], h[V / 2];
                get(X, i, a);
                get(DH, i, h);
                load2(w_pre + vec * V, w);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    h[e] = mul2(h[e], rx2);
                    a_pre[i][e] = fma2(h[e], a[e], a_pre[i][e]);
                    tot[i][e] = fma2(a[e], cx2, fma2(h[e], w[e], tot[i][e]));
                }
            }
            if (in && pass_on) store2(static_cast<T*>(p.dx) + at, tot[i]);
            if (in) {
                uint64_t rs[V / 2], a[V / 2], g[V / 2];
                const uint64_t one = two(1.f, 1.f), r2 = two(rr[i], rr[i]);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) rs[e] = one;
                if (KEEP || p.res_scale) load2(res_scale + vec * V, rs);
                load2(w_post + (whole ? vec : vec & (lanes - 1)) * V, w);
                get(Y, i, a);
                if (ACT != NO_GATE) get(GATE, i, g);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const uint64_t yn = mul2(a[e], r2), n = mul2(yn, w[e]);
                    uint64_t da = tot[i][e];              // total act
                    if (ACT != NO_GATE) {
                        float t0, t1;
                        apart(g[e], t0, t1);
                        const uint64_t q = two(sigmoid<T>(t0), sigmoid<T>(t1));
                        const uint64_t act = ACT == SILU ? mul2(g[e], q) : q;
                        // act' = act (1 - q), for silu + q
                        uint64_t slope = mul2(act, sub2(one, q));
                        if (ACT == SILU) slope = add2(slope, q);
                        g[e] = mul2(mul2(da, rs[e]), mul2(n, slope));
                        da = mul2(da, act);
                    }
                    a_res[i][e] = fma2(da, n, a_res[i][e]);
                    da = mul2(da, rs[e]);
                    a_post[i][e] = fma2(da, yn, a_post[i][e]);
                    tot[i][e] = mul2(da, w[e]);           // dn from here on
                    part = fma2(tot[i][e], a[e], part);
                }
                if (ACT != NO_GATE) store2(static_cast<T*>(p.dgate) + at, g);
            }
            if (whole) {
                s2[0] += sum2(part);
            } else {
                float pt[1] = {sum2(part)};
                lane_sum(pt, lanes);
                cc[i] = pt[0] * inv_group;
            }
        }
        if (whole) {
            row_sum(s2, buf, warps, 1);
#pragma unroll
            for (int i = 0; i < VPT; ++i) cc[i] = s2[0] * inv_row;
        } else if (sums && warps > 1) {
            row_wait();   // the next row writes the sums this row has read
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = vec0 + i * width;
            if (!FULL && vec >= vecs) continue;
            uint64_t a[V / 2];
            get(Y, i, a);
            const float c = -cc[i] * rr[i] * rr[i] * rr[i];
            const uint64_t c2 = two(c, c), r2 = two(rr[i], rr[i]);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) tot[i][e] = fma2(a[e], c2, mul2(r2, tot[i][e]));
            store2(static_cast<T*>(p.dy) + (size_t)row * D + (size_t)vec * V, tot[i]);
        }
        if (RING && ++stage == depth) stage = 0;
    }
    let_follow();
    if (RING) copies_done(0);
    __syncthreads();   // the ring's room takes the sums

    // This block's sums: threadIdx.y groups in order, then one part per block.
    // The part of dw_post holds one value per channel of a group: where a group
    // is a head, its heads are added here, in order.
    float* dyn = reinterpret_cast<float*>(dyn4);   // [tile]
    const int col0 = blockIdx.y * tile, count = vecs * V - col0;
    float* mine = p.partial + (size_t)blockIdx.x * 3 * p.D;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
        if (which == 1 && !p.res_scale) continue;
        if (which == 2 && !p.w_pre) continue;
        for (unsigned k = 0; k < blockDim.y; ++k) {
            if (threadIdx.y == k) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int vec = vec0 + i * width;
                    if (vec >= vecs) continue;
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        float v0, v1;
                        apart(which == 0   ? a_post[i][e / 2]
                              : which == 1 ? a_res[i][e / 2]
                                           : a_pre[i][e / 2],
                              v0, v1);
                        float* at = dyn + vec * V + e - col0;
                        at[0] = k ? at[0] + v0 : v0;
                        at[1] = k ? at[1] + v1 : v1;
                    }
                }
            }
            __syncthreads();
        }
        if (which == 0 && !whole) {
            for (int c = flat; c < p.group; c += all) {
                float v = dyn[c];
                for (int at = c + p.group; at < count; at += p.group) v += dyn[at];
                mine[blockIdx.y * p.group + c] = v;
            }
        } else {
            for (int c = flat; c < count; c += all) mine[which * p.D + col0 + c] = dyn[c];
        }
        __syncthreads();
    }
}

// One block per 32 columns of one of the three sums: 128 rows of 8 threads take
// the parts in turn, four columns a thread; rows are added in the order of a
// fixed tree.  dw_post of heads has a part per tile too.
__global__ void __launch_bounds__(1024) block_norm_sums_kernel(BlockNorm p, int parts, int tiles) {
    __shared__ float4 buf[32][8];
    wait_before();
    const int which = blockIdx.y;
    float* dst = which == 0 ? p.dw_post : which == 1 ? p.dres_scale : p.dw_pre;
    const int width = which == 0 ? p.group : p.D;
    const int per = which == 0 && p.group != p.D ? tiles : 1;
    if (!dst || blockIdx.x * 32 >= width) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 7) * 4, n = parts * per;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < width) {
#pragma unroll 8
        for (int k = threadIdx.x >> 3; k < n; k += 128) {
            const float4 v = *reinterpret_cast<const float4*>(
                p.partial + ((size_t)(k / per) * 3 + which) * p.D + (k % per) * width + c);
            s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
        }
    }
    auto add_rows = [&]() {      // the four rows of a warp
#pragma unroll
        for (int m = 8; m < 32; m <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], m);
    };
    add_rows();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane < 8) buf[warp][lane] = make_float4(s[0], s[1], s[2], s[3]);
    __syncthreads();
    if (warp > 0) return;
    s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
    for (int k = lane >> 3; k < 32; k += 4) {
        const float4 v = buf[k][lane & 7];
        s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
    }
    add_rows();
    if (lane < 8 && c < width) *reinterpret_cast<float4*>(dst + c) = make_float4(s[0], s[1], s[2], s[3]);
}

struct Shape {
    dim3 block;
    int vpt;
    int tile;    // columns per block
    int tiles;
};

// Up to `most` threads on a row while two vectors a thread are enough, then 512;
// short rows share a block of 128 threads.  Where no sum runs over the row
// (heads, no pre norm) a wide one is cut into tiles, blocks of their own.
Shape shape_of(int32_t D, bool coupled, int most) {
    Shape s;
    s.tile = coupled || D <= TILE ? D : TILE;
    s.tiles = (D + s.tile - 1) / s.tile;
    const int vecs = s.tile / V;
    s.vpt = vecs <= most ? 1 : vecs <= 1024 ? 2 : 4;
    const int tx = ((vecs + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    s.block = dim3(tx, tx >= 128 ? 1 : 128 / tx);
    return s;
}

constexpr int BACKWARD_THREADS = 256;
constexpr size_t RING_HALF = 110 * 1024, RING_ALL = 220 * 1024;
// What a block may have beside `buf`, alone on its SM and as one of two.
constexpr size_t ROOM_ALL = 232448 - SUMS * sizeof(float), ROOM_HALF = 110 * 1024;

// The backward's shape.  A ring of up to 3 rows in half of an SM's shared memory,
// of 2 in all of it.  With every part there the weights stay beside a ring of 2
// wherever that has room (up to 7,168 columns of bf16, 4,096 of fp32), and two rows share a
// block, and the weights, where an SM would hold one block of one row: bf16, 3,584 columns
// 60 -> 55 us, 4,096 64 -> 60; not where it holds two, 2,048 37 -> 43.
struct BackwardShape {
    Shape s;
    int stages;
    bool full, keep;
    size_t smem;
};

BackwardShape backward_shape(int32_t D, bool coupled, bool all, int bytes) {
    BackwardShape b;
    b.s = shape_of(D, coupled, BACKWARD_THREADS);
    Shape& s = b.s;
    const size_t one = (size_t)TENSORS * s.vpt * s.block.x * V * bytes, row = one * s.block.y;
    const size_t sums = (size_t)s.tile * sizeof(float);
    b.stages = 3 * row <= RING_HALF ? 3 : 2 * row <= RING_ALL ? 2 : 0;
    b.full = s.tiles * s.tile == D && s.tile == (int)s.block.x * s.vpt * V;
    b.smem = b.stages * row > sums ? b.stages * row : sums;
    b.keep = all && s.vpt <= 2 && 2 * row + 3 * sums <= ROOM_ALL;
    if (b.keep) {
        b.stages = 2;
        if (2 * row + 3 * sums > ROOM_HALF && s.block.y == 1 && 2 * s.block.x <= MAX_THREADS &&
            4 * one + 3 * sums <= ROOM_ALL) {
            s.block.y = 2;
        }
        b.smem = 2 * one * s.block.y + 3 * sums;
    }
    return b;
}

bool coupled(const BlockNorm& p) { return p.group == p.D || p.w_pre; }

template <typename T>
cudaError_t forward(const BlockNorm& p, cudaStream_t stream) {
    if (!coupled(p)) {
        const int64_t vecs = p.rows * (p.D / V), blocks = (vecs + 1023) / 1024;
        if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
        block_norm_heads_kernel<T><<<(unsigned)blocks, 256, 0, stream>>>(p, vecs);
        return cudaGetLastError();
    }
    const Shape s = shape_of(p.D, true, 512);
    const int threads = s.block.x * s.block.y;
    const int64_t rows = (p.rows + s.block.y - 1) / s.block.y, most = 152 * (1024 / threads);
    const unsigned grid = (unsigned)(rows < most ? rows : most);
    switch (s.vpt) {
        case 1: block_norm_kernel<T, 1><<<grid, s.block, 0, stream>>>(p); break;
        case 2: block_norm_kernel<T, 2><<<grid, s.block, 0, stream>>>(p); break;
        default: block_norm_kernel<T, 4><<<grid, s.block, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

// The backward's blocks along the rows: what keeps 152 SMs busy, fewer where
// there are fewer rows.
int parts_of(const Shape& s, int64_t rows, size_t smem = 0) {
    const int threads = s.block.x * s.block.y;
    const int most = 152 * (smem > ROOM_HALF ? 1 : threads <= 128 ? 4 : threads <= 256 ? 2 : 1);
    const int64_t blocks = (rows + s.block.y - 1) / s.block.y;
    return (int)(blocks < most ? (blocks < 1 ? 1 : blocks) : most);
}

template <typename T>
cudaError_t backward(const BlockNorm& p, cudaStream_t stream) {
    const BackwardShape b = backward_shape(
        p.D, coupled(p), p.group == p.D && p.w_pre && p.dx_out && p.dx, sizeof(T));
    const Shape& s = b.s;
    int parts = block_norm_parts(p.rows, p.D);
    if (b.keep) parts = std::min(parts, parts_of(s, p.rows, b.smem));
    const dim3 grid(parts, s.tiles);
    cudaError_t err = cudaSuccess;
    auto launch = [&](auto kernel) {
        // (without the attribute a block has 48 KB, the kernel's own buffer among them)
        if (b.smem + SUMS * sizeof(float) > 48 * 1024) {
            err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)b.smem);
        }
        if (err == cudaSuccess) kernel<<<grid, s.block, b.smem, stream>>>(p, s.tile, b.stages);
    };
    auto with_gate = [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (b.keep && s.vpt == 1) {
            if (b.full) launch(block_norm_backward_kernel<T, 1, ACT, true, true, true>);
            else launch(block_norm_backward_kernel<T, 1, ACT, true, false, true>);
        } else if (b.keep) {
            if (b.full) launch(block_norm_backward_kernel<T, 2, ACT, true, true, true>);
            else launch(block_norm_backward_kernel<T, 2, ACT, true, false, true>);
        } else if (b.stages == 0) {
            launch(block_norm_backward_kernel<T, 4, ACT, false, false>);
        } else if (s.vpt == 1) {
            if (b.full) launch(block_norm_backward_kernel<T, 1, ACT, true, true>);
            else launch(block_norm_backward_kernel<T, 1, ACT, true, false>);
        } else if (s.vpt == 2) {
            if (b.full) launch(block_norm_backward_kernel<T, 2, ACT, true, true>);
            else launch(block_norm_backward_kernel<T, 2, ACT, true, false>);
        } else if constexpr (sizeof(T) == 2) {   // (fp32 rows that wide have no ring)
            launch(block_norm_backward_kernel<T, 4, ACT, true, false>);
        }
    };
    if (!p.gate) {
        with_gate(std::integral_constant<int, NO_GATE>());
    } else if (p.silu) {
        with_gate(std::integral_constant<int, SILU>());
    } else {
        with_gate(std::integral_constant<int, SIGMOID>());
    }
    if (err == cudaSuccess) err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return launch_follower(block_norm_sums_kernel, dim3((p.D + 31) / 32, 3), 1024, 0, stream, p,
                           parts, s.tiles);
}

}  // namespace

// Room for the sums of the most blocks that any type takes.
int block_norm_parts(int64_t rows, int32_t D) {
    return parts_of(shape_of(D, true, BACKWARD_THREADS), rows);
}

cudaError_t launch_block_norm(const BlockNorm& p, int dtype, cudaStream_t stream) {
    return dtype == 0 ? forward<float>(p, stream) : forward<__nv_bfloat16>(p, stream);
}

cudaError_t launch_block_norm_backward(const BlockNorm& p, int dtype, cudaStream_t stream) {
    return dtype == 0 ? backward<float>(p, stream) : backward<__nv_bfloat16>(p, stream);
}

}  // namespace kda
