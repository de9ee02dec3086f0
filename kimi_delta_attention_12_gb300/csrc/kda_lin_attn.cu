// kda_lin_attn.cu -- decayed linear attention on the CUDA cores (fp32
// arithmetic) for every type and head size, and its decode step.
//
// A pass walks a segment of a sequence in chunks of C = 32 tokens with the
// state in shared memory.  With a = e^g, rows i, j of a chunk of c tokens and
// the state S before it (forward in time):
//     out_i = sum_{j <= i} a^{i-j} (x_i . y_j) z_j + a^{i+1} S^T x_i
//     S'    = a^c S + sum_j a^{c-1-j} y_j z_j^T
// A CTA owns 32 of the dz columns of one (segment, head): state columns do
// not mix, only the products x_i . y_j are formed again in each slice.
// A sequence that is cut into segments is walked twice: once for the state
// that each segment adds, and, after that, for the outputs, where a segment
// starts from the state that a scan over the segments left for it.
//
// The products keep fp32 operands, so they are the CUDA cores'; what bounds them
// is shared memory, which each multiply-add reads: 78 % of its cycles in the
// outputs' passes, 55 % of the issue slots, 7 % of the memory's rate.  Chunks of 32
// keep a quarter of X Y^T in 16 registers a thread (4 x 4 tiles: 16 multiply-adds
// for two 16-byte reads), and slices of 32 columns leave room for two CTAs an SM.
// Backward of 3,602 tokens in 5 sequences, 8 heads, 64 x 128 wide, fp32: 226 us
// (45 the segments' states, 8 the scan, 178 the outputs, each brought on while the
// one before ends); with one tile row a thread, longer segments and a launch for each
// gradient it had taken 1,520.
#include "kda_lin.h"

#include <cuda_bf16.h>
#include <limits.h>
#include <string.h>

#include "kda_follow.cuh"
#include "kda_lin.cuh"
#include "kda_packed.cuh"

namespace kda {
namespace {

constexpr int C = 32;        // tokens per chunk
constexpr int SLICE = 32;    // state columns per CTA
constexpr int THREADS = 256;

__device__ __forceinline__ float4 load4(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                       __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) {
    *reinterpret_cast<float4*>(p) = v;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 r;
    r.x = *reinterpret_cast<const uint32_t*>(&a);
    r.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = r;
}

constexpr int PLD = C + 4;   // row of a 32 x 32 tile of products

// fp32 rows come by asynchronous copies, a chunk ahead; bf16 ones are converted on
// their way through registers and have one stage.
template <typename T>
constexpr int STAGES = sizeof(T) == 4 ? 2 : 1;
template <int DX>
constexpr int STAGE_FLOATS = 2 * C * (DX + 4) + C * SLICE;   // X, Y, Z

template <typename T, int DX>
constexpr size_t pass_smem_bytes() {
    return sizeof(float) *
           (STAGES<T> * STAGE_FLOATS<DX> + 4 * C * PLD + DX * SLICE + (C + 4));
}

// Four values to shared memory, zeros instead unless `live`.
__device__ __forceinline__ void copy4(float* dst, const float* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(float* dst, const __nv_bfloat16* src, bool live) {
    store4(dst, live ? load4(src) : make_float4(0.f, 0.f, 0.f, 0.f));
}

// 4 values at the thread's rows of a state: row d of [dx][dz], or of a turned one.
__device__ __forceinline__ float4 state_at(const float* st, int d, int c, int dx, int dz,
                                           int turned) {
    if (!turned) return load4(st + (size_t)d * dz + c);
    return make_float4(st[(size_t)c * dx + d], st[(size_t)(c + 1) * dx + d],
                       st[(size_t)(c + 2) * dx + d], st[(size_t)(c + 3) * dx + d]);
}

__device__ __forceinline__ void add_scaled(float4& acc, float w, float4 v) {
    acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
}

// acc[i][j] += a row of 4 values times b's: the products of 4 rows with 4 rows
// over 4 summed values, in pairs.
__device__ __forceinline__ void dot4(uint64_t (&acc)[4][4], const float4 (&a)[4],
                                     const float4 (&b)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = fma2(two(a[i].z, a[i].w), two(b[j].z, b[j].w),
                             fma2(two(a[i].x, a[i].y), two(b[j].x, b[j].y), acc[i][j]));
}

// acc[i] += sum over 4 rows k of a[i][k] b[k].
__device__ __forceinline__ void mul4(float4 (&acc)[4], const float4 (&a)[4], const float4 (&b)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        add_scaled(acc[i], a[i].x, b[0]);
        add_scaled(acc[i], a[i].y, b[1]);
        add_scaled(acc[i], a[i].z, b[2]);
        add_scaled(acc[i], a[i].w, b[3]);
    }
}

// STATES: only the state that the segment adds, into seg_states.
//
// The two 32 x 32 products (x . y, and the outputs) are formed by four groups of
// 64 threads, each over a quarter of the summed index in 4 x 4 tiles (16
// multiply-adds for every two 16-byte reads of shared memory), and the quarters
// added in order; the state's product has 4 columns and dx / 32 rows a thread.
template <typename T, int DX, bool STATES>
__device__ __forceinline__ void pass(const LinPass& p, uint32_t block) {
    constexpr int LD = DX + 4, ROWS = DX / 32;
    extern __shared__ float4 smem4[];
    float* stages = reinterpret_cast<float*>(smem4);
    float* P = stages + STAGES<T> * STAGE_FLOATS<DX>;   // [4][C][PLD]
    float* S = P + 4 * C * PLD;       // [DX][SLICE]
    float* lam = S + DX * SLICE;      // a^0 .. a^C

    const int tid = threadIdx.x, dz = p.dz, slices = dz / SLICE;
    const int col0 = (int)(block % slices) * SLICE;
    const int64_t rest = block / slices;
    const int h = (int)(rest % p.H);
    const lin::Segment sg = lin::find_segment(p.cu_seqlens, p.N, p.total_T, p.seg_len, p.reverse,
                                              rest / p.H);
    if (sg.n < 0 || (STATES && sg.j + 1 >= sg.count)) return;
    const float g = p.log_decay[h];
    if (tid <= C) lam[tid] = lin::decay_pow(g, tid);

    const size_t state_floats = (size_t)DX * dz;
    const int64_t rows = lin::seg_rows(p.total_T, p.seg_len);
    const int c4 = (tid & 7) * 4, d0 = (tid / 8) * ROWS;   // the thread's part of the state
    float4 st[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) st[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!STATES) {
        // the state before the segment: the initial one, or what the scan left
        if (sg.j > 0) {
            if (sg.u + sg.j - 1 < rows) {      // (else a malformed cu_seqlens)
                const float* s0 =
                    p.seg_states + ((sg.u + sg.j - 1) * (int64_t)p.H + h) * state_floats;
#pragma unroll
                for (int i = 0; i < ROWS; ++i)
                    st[i] = load4(s0 + (size_t)(d0 + i) * dz + col0 + c4);
            }
        } else if (p.state_in) {
            const float* s0 = p.state_in + ((size_t)sg.n * p.H + h) * state_floats;
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                st[i] = state_at(s0, d0 + i, col0 + c4, DX, dz, p.state_in_turned);
        }
    }

    const T* x = static_cast<const T*>(p.x);
    const T* y = static_cast<const T*>(p.y);
    const T* z = static_cast<const T*>(p.z);
    T* out = static_cast<T*>(p.out);
    // group of the thread, and its tile's rows r + 8 i and columns q + 8 j (of
    // x . y) or 4 q .. 4 q + 3 (of the outputs)
    const int grp = tid / 64, r = (tid / 8) & 7, q = tid & 7;
    const int64_t chunks = (sg.t1 - sg.t0 + C - 1) / C;
    auto first = [&](int64_t ci) { return sg.t0 + (p.reverse ? chunks - 1 - ci : ci) * C; };
    auto load_chunk = [&](int64_t ci) {
        float* X = stages + (ci % STAGES<T>) * STAGE_FLOATS<DX>;
        float *Y = X + C * LD, *Z = Y + C * LD;
        const int64_t c0 = first(ci);
        const int len = (int)(sg.t1 - c0 < C ? sg.t1 - c0 : C);
#pragma unroll
        for (int k = 0; k < C * DX / 4 / THREADS; ++k) {
            const int i = tid + k * THREADS, row = i / (DX / 4), d = (i % (DX / 4)) * 4;
            const bool live = row < len;
            const size_t at = ((size_t)(c0 + (live ? row : 0)) * p.H + h) * DX + d;
            if (!STATES) copy4(X + row * LD + d, x + at, live);
            copy4(Y + row * LD + d, y + at, live);
        }
        const int row = tid / 8;
        const bool live = row < len;
        copy4(Z + row * SLICE + c4,
              z + ((size_t)(c0 + (live ? row : 0)) * p.H + h) * dz + col0 + c4, live);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (STAGES<T> == 2 && chunks > 0) load_chunk(0);
    if (STATES) __syncthreads();   // lam
    for (int64_t ci = 0; ci < chunks; ++ci) {
        const int64_t c0 = first(ci);
        const int len = (int)(sg.t1 - c0 < C ? sg.t1 - c0 : C);
        const float* X = stages + (ci % STAGES<T>) * STAGE_FLOATS<DX>;
        const float* Y = X + C * LD;
        float* Z = stages + (ci % STAGES<T>) * STAGE_FLOATS<DX> + 2 * C * LD;
        // the thread's four values of Z, which it has copied, get their weight in the state;
        // rows past the end none (a growing decay's power there may be infinite)
        auto weigh = [&] {
            const int s = tid / 8;
            const float w = s < len ? lam[p.reverse ? s + 1 : len - 1 - s] * p.kv_scale : 0.0f;
            float4 v = load4(Z + s * SLICE + c4);
            v.x *= w; v.y *= w; v.z *= w; v.w *= w;
            store4(Z + s * SLICE + c4, v);
        };
        if (STAGES<T> == 1) {
            load_chunk(ci);
        } else if (ci + 1 < chunks) {
            load_chunk(ci + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        if (!STATES) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) store4(S + (d0 + i) * SLICE + c4, st[i]);
        } else {
            weigh();
        }
        __syncthreads();
        if (!STATES) {
            {
                uint64_t acc[4][4] = {};
#pragma unroll 4
                for (int d = grp * (DX / 4); d < (grp + 1) * (DX / 4); d += 4) {
                    float4 a[4], b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i] = load4(X + (r + 8 * i) * LD + d);
                        b[i] = load4(Y + (q + 8 * i) * LD + d);
                    }
                    dot4(acc, a, b);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        P[(grp * C + r + 8 * i) * PLD + q + 8 * j] = sum2(acc[i][j]);
            }
            __syncthreads();
            {
                // the quarters together, masked and weighted
                const int t = tid / 8;
                float4 v = load4(P + t * PLD + c4);
#pragma unroll
                for (int k = 1; k < 4; ++k) {
                    const float4 w = load4(P + (k * C + t) * PLD + c4);
                    v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
                }
                float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int s = c4 + j, dist = p.reverse ? s - t : t - s;
                    e[j] = dist >= 0 && s < len ? e[j] * (lam[dist & (C - 1)] * p.kv_scale) : 0.0f;
                }
                store4(P + t * PLD + c4, make_float4(e[0], e[1], e[2], e[3]));
            }
            __syncthreads();
            {
                float4 intra[4], inter[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) intra[i] = inter[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int s = 8 * grp; s < 8 * grp + 8; s += 4) {
                    float4 a[4], b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i] = load4(P + (r + 8 * i) * PLD + s);
                        b[i] = load4(Z + (s + i) * SLICE + 4 * q);
                    }
                    mul4(intra, a, b);
                }
#pragma unroll 4
                for (int d = grp * (DX / 4); d < (grp + 1) * (DX / 4); d += 4) {
                    float4 a[4], b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i] = load4(X + (r + 8 * i) * LD + d);
                        b[i] = load4(S + (d + i) * SLICE + 4 * q);
                    }
                    mul4(inter, a, b);
                }
                __syncthreads();   // P is read; its room takes the quarters of the outputs
                weigh();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = r + 8 * i;
                    const float f = t < len ? lam[p.reverse ? len - 1 - t : t + 1] : 0.0f;
                    add_scaled(intra[i], f, inter[i]);
                    store4(P + (grp * C + t) * PLD + 4 * q, intra[i]);
                }
            }
            __syncthreads();
            const int t = tid / 8;
            if (t < len) {
                float4 v = load4(P + t * PLD + c4);
#pragma unroll
                for (int k = 1; k < 4; ++k) {
                    const float4 w = load4(P + (k * C + t) * PLD + c4);
                    v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
                }
                const float m = p.out_scale;
                store4(out + ((size_t)(c0 + t) * p.H + h) * dz + col0 + c4,
                       make_float4(m * v.x, m * v.y, m * v.z, m * v.w));
            }
        }
        const float f = lam[len];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            st[i].x *= f; st[i].y *= f; st[i].z *= f; st[i].w *= f;
        }
#pragma unroll 8
        for (int s = 0; s < C; ++s) {     // rows past the end are zeros
            const float4 v = load4(Z + s * SLICE + c4);
            float k[ROWS];
            if (ROWS == 4) {
                const float4 k4 = load4(Y + s * LD + d0);
                k[0] = k4.x; k[1 % ROWS] = k4.y; k[2 % ROWS] = k4.z; k[3 % ROWS] = k4.w;
            } else {
#pragma unroll
                for (int i = 0; i < ROWS; ++i) k[i] = Y[s * LD + d0 + i];
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) add_scaled(st[i], k[i], v);
        }
        __syncthreads();   // the next chunk's rows overwrite this one's
    }

    float* dst = nullptr;
    if (STATES) {
        if (sg.u + sg.j < rows)
            dst = p.seg_states + ((sg.u + sg.j) * (int64_t)p.H + h) * state_floats;
    } else if (p.state_out && sg.j + 1 == sg.count) {
        dst = p.state_out + ((size_t)sg.n * p.H + h) * state_floats;
    }
    if (dst) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) store4(dst + (size_t)(d0 + i) * dz + col0 + c4, st[i]);
    }
}

// Up to three passes of one call, one after another in the grid: the blocks of the
// next fill the SMs that the last round of the one before leaves idle.
struct Passes {
    LinPass p[3];
    uint32_t end[3];   // blocks of the passes up to this one
};

template <typename T, bool STATES>
__global__ void __launch_bounds__(THREADS, 2)
lin_passes_kernel(const __grid_constant__ Passes jobs) {
    const int k = blockIdx.x < jobs.end[0] ? 0 : blockIdx.x < jobs.end[1] ? 1 : 2;
    const LinPass& p = jobs.p[k];
    const uint32_t block = blockIdx.x - (k > 0 ? jobs.end[k - 1] : 0);
    if (STATES) let_follow();
    else wait_before();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;   // no wait here can run out
    if (p.dx == 32) pass<T, 32, STATES>(p, block);
    else if (p.dx == 64) pass<T, 64, STATES>(p, block);
    else pass<T, 128, STATES>(p, block);
}

template <typename T>
size_t pass_smem(int dx) {
    return dx == 32   ? pass_smem_bytes<T, 32>()
           : dx == 64 ? pass_smem_bytes<T, 64>()
                      : pass_smem_bytes<T, 128>();
}

template <typename T, bool STATES>
cudaError_t launch_passes(const LinPass* passes, int n, bool follows, cudaStream_t stream) {
    Passes jobs;
    memset(&jobs, 0, sizeof(jobs));
    int64_t grid = 0;
    size_t smem = 0;
    for (int i = 0; i < 3; ++i) {
        if (i < n) {
            const LinPass& p = jobs.p[i] = passes[i];
            const int64_t most = (int64_t)p.total_T / p.seg_len;   // segments that are not a last one
            if (!STATES || most > 0) grid += (most + p.N) * p.H * (p.dz / SLICE);
            const size_t need = pass_smem<T>(p.dx);
            if (need > smem) smem = need;
        }
        if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
        jobs.end[i] = (uint32_t)grid;
    }
    if (grid == 0) return cudaSuccess;
    auto* kernel = lin_passes_kernel<T, STATES>;
    const cudaError_t err =
        smem <= 48 * 1024
            ? cudaSuccess
            : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    if (follows) return launch_follower(kernel, (unsigned)grid, THREADS, smem, stream, jobs);
    kernel<<<(unsigned)grid, THREADS, smem, stream>>>(jobs);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run_passes(const LinPass* passes, int n, cudaStream_t stream) {
    bool cut = false;
    for (int i = 0; i < n; ++i) {
        const int32_t dx = passes[i].dx;
        if (dx != 32 && dx != 64 && dx != 128) return cudaErrorInvalidValue;
        cut = cut || passes[i].total_T >= passes[i].seg_len;
    }
    cudaError_t err = cudaSuccess;
    if (cut) err = launch_passes<T, true>(passes, n, false, stream);
    if (cut && err == cudaSuccess) err = launch_lin_scan(passes, n, stream);
    if (err == cudaSuccess) err = launch_passes<T, false>(passes, n, cut, stream);
    return err;
}

// ------------------------------------------------------ states between segments
// S_{j+1} = a^{tokens of segment j} S_j + (what segment j adds), one float4 of the
// state per thread, the rows of four segments on their way at once.
constexpr int SCAN_THREADS = 128;

struct Scan {
    LinPass p[3];
};

__global__ void __launch_bounds__(SCAN_THREADS) lin_scan_kernel(const __grid_constant__ Scan scan) {
    let_follow();
    wait_before();
    const LinPass& p = scan.p[blockIdx.y];
    const int per = p.dx * p.dz / 4 / SCAN_THREADS;       // blocks of one state
    const int64_t pair = blockIdx.x / per;
    const int n = (int)(pair / p.H), h = (int)(pair % p.H);
    const int at = (blockIdx.x % per) * SCAN_THREADS + threadIdx.x;
    const lin::Segment sg = lin::first_segment(p.cu_seqlens, p.N, p.total_T, p.seg_len, p.reverse,
                                               n);
    if (sg.count < 2 || (p.lead > 0 && sg.count <= p.lead)) return;
    const float g = p.log_decay[h];
    const int64_t rows = lin::seg_rows(p.total_T, p.seg_len);
    const size_t state4 = (size_t)p.dx * p.dz / 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.state_in) {
        const float* s0 = p.state_in + (size_t)pair * p.dx * p.dz;
        const int d = at * 4 / p.dz, c = at * 4 % p.dz;
        s = state_at(s0, d, c, p.dx, p.dz, p.state_in_turned);
    }
    float4* u = reinterpret_cast<float4*>(p.seg_states) + at;
    const int used = p.lead > 0 ? p.lead : sg.count - 1;
    const int last = (int)(rows - sg.u < used ? rows - sg.u : used);
    for (int j = 0; j < last; j += 4) {
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j + k < last) v[k] = u[((sg.u + j + k) * (int64_t)p.H + h) * state4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (j + k >= last) break;
            int64_t a, b;
            lin::seg_tokens(sg, j + k, p.seg_len, p.reverse, a, b);
            const float f = lin::decay_pow(g, b - a);
            s.x = f * s.x + v[k].x;
            s.y = f * s.y + v[k].y;
            s.z = f * s.z + v[k].z;
            s.w = f * s.w + v[k].w;
            u[((sg.u + j + k) * (int64_t)p.H + h) * state4] = s;
        }
    }
}

// ------------------------------------------------------------------ decode
// S = a S + k v^T, o = scale S^T q: the state is read and written once, so the
// step is bound by 8 d_k d_v bytes per (row, head).  A CTA takes 32 columns:
// 8 lanes cover a 128-byte piece of a state row, so that every warp request is
// four full lines, and each thread has its d_k / 16 rows in flight at once.  256
// rows of 96 heads, 128 x 128, bf16: 466 us, 6.96 TB/s (1.02 of a plain copy's rate);
// one row of 32 heads: 4 us on the device, which is a launch and one trip to memory.
constexpr int DEC_THREADS = 128;

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(DEC_THREADS) lin_decode_kernel(LinDecode p) {
    constexpr int STEP = DEC_THREADS / 8, ROWS = DK / STEP, slices = DV / 32;
    __shared__ float sq[DK], sk[DK];
    __shared__ float4 part[DEC_THREADS / 32][8];
    const int tid = threadIdx.x, c = (blockIdx.x % slices) * 32 + (tid & 7) * 4;
    const int64_t bh = blockIdx.x / slices;
    const int h = (int)(bh % p.H);
    const int64_t b = bh / p.H;
    const int64_t slot = p.slots ? p.slots[b] : b;
    T* o = static_cast<T*>(p.o) + bh * DV;
    if (slot < 0 || slot >= p.pool_size) {
        if (tid < 8) {
            const float nan = __int_as_float(0x7fffffff);
            store4(o + c, make_float4(nan, nan, nan, nan));
        }
        return;
    }
    float* st = p.state + (slot * p.H + h) * (int64_t)(DK * DV) + c;
    float4 s[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        s[i] = __ldcs(reinterpret_cast<const float4*>(st + (tid / 8 + STEP * i) * DV));
    const float4 v = load4(static_cast<const T*>(p.v) + bh * DV + c);
    if (tid < DK / 4) store4(sq + 4 * tid, load4(static_cast<const T*>(p.q) + bh * DK + 4 * tid));
    else if (tid >= 64 && tid < 64 + DK / 4)
        store4(sk + 4 * (tid - 64), load4(static_cast<const T*>(p.k) + bh * DK + 4 * (tid - 64)));
    const float a = lin::decay_pow(p.log_decay[h], 1);
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int d = tid / 8 + STEP * i;
        const float k = sk[d], q = sq[d];
        s[i].x = a * s[i].x + k * v.x;
        s[i].y = a * s[i].y + k * v.y;
        s[i].z = a * s[i].z + k * v.z;
        s[i].w = a * s[i].w + k * v.w;
        __stcs(reinterpret_cast<float4*>(st + d * DV), s[i]);
        acc.x += q * s[i].x; acc.y += q * s[i].y; acc.z += q * s[i].z; acc.w += q * s[i].w;
    }
#pragma unroll
    for (int m = 8; m < 32; m <<= 1) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, m);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, m);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, m);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, m);
    }
    if ((tid & 31) < 8) part[tid / 32][tid & 7] = acc;
    __syncthreads();
    if (tid < 8) {
        float4 r = part[0][tid];
#pragma unroll
        for (int w = 1; w < DEC_THREADS / 32; ++w) {
            r.x += part[w][tid].x; r.y += part[w][tid].y;
            r.z += part[w][tid].z; r.w += part[w][tid].w;
        }
        store4(o + c, make_float4(p.scale * r.x, p.scale * r.y, p.scale * r.z, p.scale * r.w));
    }
}

template <typename T, int DK, int DV>
cudaError_t launch_decode(const LinDecode& p, cudaStream_t stream) {
    const int64_t grid = (int64_t)p.B * p.H * (DV / 32);
    if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
    lin_decode_kernel<T, DK, DV><<<(unsigned)grid, DEC_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t decode_dv(const LinDecode& p, int d_v, cudaStream_t stream) {
    switch (d_v) {
        case 32: return launch_decode<T, DK, 32>(p, stream);
        case 64: return launch_decode<T, DK, 64>(p, stream);
        case 128: return launch_decode<T, DK, 128>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <typename T>
cudaError_t decode_dk(const LinDecode& p, int d_k, int d_v, cudaStream_t stream) {
    switch (d_k) {
        case 32: return decode_dv<T, 32>(p, d_v, stream);
        case 64: return decode_dv<T, 64>(p, d_v, stream);
        case 128: return decode_dv<T, 128>(p, d_v, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

LinCut lin_cut(int32_t N, int32_t total_T, int32_t H, int ctas_per_pair, int ctas_per_sm, int sms) {
    constexpr int64_t grain = 128;
    if (sms <= 0) sms = 152;   // no device to ask: sizes for a whole GB300
    const int64_t pairs = (int64_t)N * H * ctas_per_pair;
    const int64_t cuts = (int64_t)sms * ctas_per_sm / pairs;
    if (cuts < 2) return {INT32_MAX / grain * grain, 0};
    const int64_t len = ((int64_t)total_T + N * cuts - 1) / (N * cuts);
    const int64_t seg = (len + grain - 1) / grain * grain;
    return {(int32_t)(seg < grain ? grain : seg), 0};
}

LinCut lin_cut_tc(int32_t N, int32_t total_T, int32_t H, int passes, int sms) {
    if (sms <= 0) sms = 152;
    const LinCut whole = lin_cut(N, total_T, H, passes, 1, sms);
    const int64_t pairs = (int64_t)N * H * passes, chunks = total_T / (128 * (int64_t)N);
    if (whole.seg_len <= total_T || pairs >= sms) return whole;
    const int64_t k = (pairs + sms - pairs - 1) / (sms - pairs), head = chunks / (k + 1);
    // A cut saves the heads' time, but their states come first (a chunk of them takes
    // about half of a chunk's time), and 152 busy SMs share the memory.  96 heads:
    // 8K tokens 203 -> 209 us, 16K 393 -> 366, 64K 1,528 -> 1,291; 112 heads: 8K 207 ->
    // 227, 32K 786 -> 748; the backward of 32 heads: 8K 205 -> 221, 16K 396 -> 393, 32K
    // 779 -> 675.
    if (k > 3 || chunks < 64 * k) return whole;
    int64_t lead = 1, best = 0;
    for (int64_t n = 1; n <= 8; ++n) {     // segments that share the SMs best; 3 chunks' start
        const int64_t time = (pairs * n + sms - 1) / sms * ((head + n - 1) / n + 3);
        if (best == 0 || time < best) {
            best = time;
            lead = n;
        }
    }
    return {(int32_t)((head + lead - 1) / lead * 128), (int32_t)lead};
}

cudaError_t launch_lin_scan(const LinPass* passes, int n, cudaStream_t stream) {
    Scan scan;
    for (int i = 0; i < n; ++i) scan.p[i] = passes[i];
    const LinPass& p = passes[0];
    const int64_t grid = (int64_t)p.N * p.H * (p.dx * p.dz / 4 / SCAN_THREADS);
    if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
    return launch_follower(lin_scan_kernel, dim3((unsigned)grid, n), SCAN_THREADS, 0, stream, scan);
}

cudaError_t launch_lin_pass(const LinPass* passes, int n, int dtype, cudaStream_t stream) {
    return dtype == 0 ? run_passes<float>(passes, n, stream)
                      : run_passes<__nv_bfloat16>(passes, n, stream);
}

cudaError_t launch_lin_decode(const LinDecode& p, int d_k, int d_v, int dtype,
                              cudaStream_t stream) {
    return dtype == 0 ? decode_dk<float>(p, d_k, d_v, stream)
                      : decode_dk<__nv_bfloat16>(p, d_k, d_v, stream);
}

}  // namespace kda
