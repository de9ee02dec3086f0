// kda_cache_write.cu -- new keys and values into the paged 8-bit cache (kda_cache_write in
// include/kda.h).  A run is what a call writes into one block: consecutive rows with rising
// slots, cut at the block's end.  Its largest value gives the scale, a power of two, so that
// dividing by it is exact, and tokens that are already in the block move to a larger scale by a
// change of exponent.
//
// Bound by HBM: bf16 2 bytes read and 1 written a value.  A run's values stay in registers
// between the maximum and the rounding, so they are read once.  A block of threads takes the
// runs that begin among `tile` rows, for one head and one of k and v: runs of more than
// kShort rows one after the other with all its threads, shorter ones one to a warp.  Which
// rows begin a run shows from the slots alone.
#include <cuda_bf16.h>

#include "kda_cache.h"
#include "kda_e4m3.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostTile = 64;
constexpr int kShort = 8;        // rows of a run that one warp takes alone

// Rows of the run that begins at row t (slot s), at most `most` (what its block has left).
__device__ __forceinline__ int run_length(const int32_t* slots, int T, int t, int s, int most,
                                          int lane) {
    int n = 1;
    while (n < most) {
        const int i = n + lane;
        const bool goes_on = i < most && t + i < T && slots[t + i] == s + i;
        const uint32_t stop = __ballot_sync(0xffffffffu, !goes_on);
        if (stop) return n + __ffs(stop) - 1;
        n += 32;
    }
    return n;
}

template <bool BF16>
__device__ __forceinline__ void values_of(const uint4& raw, float* x) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            x[i] = __uint_as_float(w[i]);
        }
    }
}

// The largest finite magnitude.
template <bool BF16>
__device__ __forceinline__ float largest_of(const uint4& raw, float best) {
    float x[BF16 ? 8 : 4];
    values_of<BF16>(raw, x);
#pragma unroll
    for (int i = 0; i < (BF16 ? 8 : 4); ++i) {
        const float a = fabsf(x[i]);
        best = a < __int_as_float(0x7f800000) ? fmaxf(best, a) : best;
    }
    return best;
}

__device__ __forceinline__ float quotient(float x, float scale, float inverse) {
    return inverse != 0.0f ? x * inverse : __fdiv_rn(x, scale);
}

// x / scale is x times its inverse, exactly, for a power of two whose inverse is a normal
// number; 0 says that it is to be divided.
__device__ __forceinline__ float exact_inverse(float scale) {
    const uint32_t bits = __float_as_uint(scale), e = bits >> 23;
    return (bits & 0x7fffffu) == 0 && e >= 1 && e <= 253 ? __uint_as_float((254 - e) << 23) : 0.0f;
}

template <bool BF16>
__device__ __forceinline__ void store_rounded(uint8_t* to, const uint4& raw, float scale,
                                              float inverse) {
    float x[BF16 ? 8 : 4];
    values_of<BF16>(raw, x);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 1); ++i) {
        const uint32_t lo = e4m3_of(quotient(x[4 * i], scale, inverse),
                                    quotient(x[4 * i + 1], scale, inverse));
        const uint32_t hi = e4m3_of(quotient(x[4 * i + 2], scale, inverse),
                                    quotient(x[4 * i + 3], scale, inverse));
        w[i] = lo | (hi << 16);
    }
    if (BF16) {
        *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint32_t*>(to) = w[0];
    }
}

// The earlier tokens of a block, 16 numbers from `at`, times `ratio`.
__device__ __forceinline__ void rescale16(uint8_t* at, float ratio) {
    uint4 raw = *reinterpret_cast<uint4*>(at);
    uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t r = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t h = j ? half2_of_e4m3_high(w[i]) : half2_of_e4m3(w[i]);
            float a, b;
            asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
                "cvt.f32.f16 %1, hi;\n\t}"
                : "=f"(a), "=f"(b)
                : "r"(h));
            r |= e4m3_of(a * ratio, b * ratio) << (16 * j);
        }
        w[i] = r;
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// One run, by 32 * W threads (`tid` among them): rows t .. t + n of head h into block b from
// place `off` on.  At most M vectors fall to a thread.
template <bool BF16, int W, int M>
__device__ __forceinline__ void write_run(const CacheWrite& p, int which, int h, int t, int n,
                                          int b, int off, int tid, float* shared) {
    constexpr int size = BF16 ? 2 : 4, per = 16 / size, threads = 32 * W;
    const int vecs = p.d / per, count = n * vecs;
    const int64_t stride = which ? p.stride[1] : p.stride[0];
    const char* x = static_cast<const char*>(which ? p.x[1] : p.x[0]) +
                    ((int64_t)t * stride + (int64_t)h * p.d) * size;
    const int64_t tile = ((int64_t)b * p.heads + h) << p.block_log2;
    uint8_t* cache = (which ? p.cache[1] : p.cache[0]) + tile * p.d;
    float* scale_at = (which ? p.scale[1] : p.scale[0]) + (int64_t)b * p.heads + h;
    const float before = off > 0 ? *scale_at : 0.0f;
    uint4 raw[M];
    float best = 0.0f;
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int u = tid + i * threads;
        if (u < count) {
            const int row = u / vecs, col = u - row * vecs;
            raw[i] = __ldcs(reinterpret_cast<const uint4*>(x + row * stride * size) + col);
        }
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
        if (tid + i * threads < count) best = largest_of<BF16>(raw[i], best);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
    if (W > 1) {
        if ((tid & 31) == 0) shared[tid >> 5] = best;
        __syncthreads();
        best = shared[0];
#pragma unroll
        for (int i = 1; i < W; ++i) best = fmaxf(best, shared[i]);
        __syncthreads();
    }
    const float fresh = e4m3_scale(best);
    const float scale = off > 0 && before > fresh ? before : fresh;
    const float inverse = exact_inverse(scale);
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int u = tid + i * threads;
        if (u < count) {
            const int row = u / vecs, col = u - row * vecs;
            store_rounded<BF16>(cache + (int64_t)(off + row) * p.d + col * per, raw[i], scale,
                                inverse);
        }
    }
    if (off > 0 && scale != before) {
        const float ratio = __fdiv_rn(before, scale);
        for (int u = tid; u < off * p.d / 16; u += threads) rescale16(cache + 16 * u, ratio);
    }
    if (W == 1) __syncwarp();
    if (tid == 0) *scale_at = scale;       // this run's threads have all read it
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(CacheWrite p, int tile) {
    __shared__ int32_t at[kMostTile];        // rows of the tile that begin a run
    __shared__ int32_t length[kMostTile];
    __shared__ float shared[kWarps];
    __shared__ int begins;
    const int h = blockIdx.y, which = blockIdx.z;
    const int t0 = blockIdx.x * tile, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int size = 1 << p.block_log2;
    const int64_t pool = (int64_t)p.num_blocks << p.block_log2;
    if (w == 0) {
        int n = 0;
        for (int base = 0; base < tile; base += 32) {
            const int i = base + lane, t = t0 + i;
            bool begin = false;
            if (i < tile && t < p.T) {
                const int32_t s = p.slots[t];
                begin = s >= 0 && s < pool &&
                        (t == 0 || (s & (size - 1)) == 0 || p.slots[t - 1] != s - 1);
            }
            const uint32_t all = __ballot_sync(0xffffffffu, begin);
            if (begin) at[n + __popc(all & ((1u << lane) - 1))] = t;
            n += __popc(all);
        }
        if (lane == 0) begins = n;
    }
    __syncthreads();
    const int n = begins;
    for (int i = w; i < n; i += kWarps) {
        const int32_t s = p.slots[at[i]];
        const int len = run_length(p.slots, p.T, at[i], s, size - (s & (size - 1)), lane);
        if (lane == 0) length[i] = len;
        if (len <= kShort) {
            write_run<BF16, 1, BF16 ? 4 : 8>(p, which, h, at[i], len, s >> p.block_log2,
                                             s & (size - 1), lane, nullptr);
        }
    }
    __syncthreads();
    for (int i = 0; i < n; ++i) {
        if (length[i] <= kShort) continue;
        const int32_t s = p.slots[at[i]];
        write_run<BF16, kWarps, BF16 ? 8 : 16>(p, which, h, at[i], length[i], s >> p.block_log2,
                                               s & (size - 1), threadIdx.x, shared);
    }
}

}  // namespace

cudaError_t launch_cache_write(const CacheWrite& p, int dtype, cudaStream_t stream) {
    const int tile = p.T <= 4096 ? 8 : kMostTile;
    const dim3 grid((p.T + tile - 1) / tile, p.heads, 2);
    auto kernel = dtype == 0 ? cache_write_kernel<false> : cache_write_kernel<true>;
    kernel<<<grid, kThreads, 0, stream>>>(p, tile);
    return cudaGetLastError();
}

}  // namespace kda
