// kda_cache_write.cu -- new keys and values into the paged 8-bit cache (kda_cache_write in
// include/kda.h).  A run is what a call writes into one block: consecutive rows with rising
// slots, cut at the block's end.  Its largest value gives the scale, a power of two, so that
// dividing by it is exact, and tokens that are already in the block move to a larger scale by a
// change of exponent.
//
// Bound by HBM: bf16 2 bytes read and 1 written a value.  A run's values stay in registers
// between the maximum and the rounding, so they are read once.  A block of threads takes the
// runs that begin among `tile` rows, for some of the heads of k and v: a run of a head goes to
// as many warps as can hold it, which wait for one another alone.  Which rows begin a run shows
// from the slots alone.  65,536 tokens of 8 heads, d = 128, bf16, blocks of 64: 66 us, 6.1 TB/s, 91 %
// of the measured copy; with all 8 warps on one run 94, with maxima of single fp32 values 118.
#include <cuda_bf16.h>

#include "kda_cache.h"
#include "kda_e4m3.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostTile = 64;
constexpr int kShort = 256;      // vectors of a run that one warp takes alone
constexpr int kBlocks = 4096;    // of threads, that a call aims at
constexpr int kFewRows = 4096;
constexpr int kWave = 640;       // blocks at once, about: four (bf16) or three for each of GB300's 152 SMs

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

// Magnitudes compare as whole numbers, bf16 ones two at a time; whether one of them is not
// finite shows at the end, and only then each is looked at.
template <bool BF16>
__device__ __forceinline__ uint32_t most_of(const uint4& raw, uint32_t best) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        best = BF16 ? __vmaxu2(best, w[i] & 0x7fff7fffu) : max(best, w[i] & 0x7fffffffu);
    }
    return best;
}

template <bool BF16>
__device__ __forceinline__ uint32_t most_finite_of(const uint4& raw, uint32_t best) {
    float x[BF16 ? 8 : 4];
    values_of<BF16>(raw, x);
#pragma unroll
    for (int i = 0; i < (BF16 ? 8 : 4); ++i) {
        const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
        best = a < 0x7f800000u ? max(best, a) : best;
    }
    return best;
}

// 1 / scale for a power of two whose inverse is a normal number: the product with it is the
// quotient, exactly.  0 says that it is to be divided.
__device__ __forceinline__ float exact_inverse(float scale) {
    const uint32_t bits = __float_as_uint(scale), e = bits >> 23;
    return (bits & 0x7fffffu) == 0 && e >= 1 && e <= 253 ? __uint_as_float((254 - e) << 23) : 0.0f;
}

template <bool BF16, bool DIVIDE>
__device__ __forceinline__ void store_rounded(uint8_t* to, const uint4& raw, float by) {
    float x[BF16 ? 8 : 4];
    values_of<BF16>(raw, x);
#pragma unroll
    for (int i = 0; i < (BF16 ? 8 : 4); ++i) x[i] = DIVIDE ? __fdiv_rn(x[i], by) : x[i] * by;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 1); ++i) {
        w[i] = e4m3_of(x[4 * i], x[4 * i + 1]) | e4m3_of(x[4 * i + 2], x[4 * i + 3]) << 16;
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

// The barrier of some warps of a block.
template <int THREADS>
__device__ __forceinline__ void meet(int barrier) {
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "n"(THREADS) : "memory");
}

// One run for one head of k or v: rows t .. t + n into block b from place `off` on.
struct Run {
    const char* x;
    int64_t stride;          // in bytes
    uint8_t* cache;          // the block's first place
    float* scale;
    int count, off;          // vectors of 16 bytes; places ahead
};

template <bool BF16>
__device__ __forceinline__ Run run_of(const CacheWrite& p, int unit, int t, int n, int32_t slot) {
    constexpr int size = BF16 ? 2 : 4;
    const bool second = unit >= p.heads;
    const int h = second ? unit - p.heads : unit;
    const int64_t at = (int64_t)(slot >> p.block_log2) * p.heads + h;
    Run r;
    r.stride = (second ? p.stride[1] : p.stride[0]) * size;
    r.x = static_cast<const char*>(second ? p.x[1] : p.x[0]) + t * r.stride + (int64_t)h * p.d * size;
    r.cache = (second ? p.cache[1] : p.cache[0]) + (at << p.block_log2) * p.d;
    r.scale = (second ? p.scale[1] : p.scale[0]) + at;
    r.count = n * p.d * size / 16;
    r.off = slot & ((1 << p.block_log2) - 1);
    return r;
}

// The run's vectors into registers, by 32 * W threads, at most M to each.
template <int W, int M>
__device__ __forceinline__ void load_run(const Run& r, int vecs_log2, int tid, uint4 (&raw)[M],
                                         float* before) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int u = tid + i * 32 * W;
        if (u < r.count) {
            const int row = u >> vecs_log2, col = u & ((1 << vecs_log2) - 1);
            raw[i] = __ldcs(reinterpret_cast<const uint4*>(r.x + row * r.stride) + col);
        }
    }
    *before = r.off > 0 ? *r.scale : 0.0f;
}

// Its scale, and its values into the cache.  shared: W words that no thread still reads;
// barrier: the W warps' own.
template <bool BF16, int W, int M>
__device__ __forceinline__ void finish_run(const Run& r, int d, int vecs_log2, int tid,
                                           const uint4 (&raw)[M], float before, uint32_t* shared,
                                           int barrier) {
    constexpr int per = BF16 ? 8 : 4;
    // the largest over the run: a bf16 magnitude in the upper half, as fp32 has it
    auto most = [&](uint32_t x) {
        x = __reduce_max_sync(0xffffffffu, x);
        if (W > 1) {
            if ((tid & 31) == 0) shared[tid >> 5] = x;
            meet<32 * W>(barrier);
            x = shared[0];
#pragma unroll
            for (int i = 1; i < W; ++i) x = max(x, shared[i]);
        }
        return x;
    };
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < M; ++i) {
        if (tid + i * 32 * W < r.count) best = most_of<BF16>(raw[i], best);
    }
    best = most(BF16 ? max(best << 16, best & 0xffff0000u) : best);
    if (best >= 0x7f800000u) {
        if (W > 1) meet<32 * W>(barrier);    // all have read `shared`
        best = 0;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            if (tid + i * 32 * W < r.count) best = most_finite_of<BF16>(raw[i], best);
        }
        best = most(best);
    }
    const float fresh = e4m3_scale(__uint_as_float(best));
    const float scale = r.off > 0 && before > fresh ? before : fresh;
    const float inverse = exact_inverse(scale);
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int u = tid + i * 32 * W;
        if (u < r.count) {
            const int row = u >> vecs_log2, col = u & ((1 << vecs_log2) - 1);
            uint8_t* to = r.cache + (r.off + row) * d + col * per;
            if (inverse != 0.0f) {
                store_rounded<BF16, false>(to, raw[i], inverse);
            } else {
                store_rounded<BF16, true>(to, raw[i], scale);
            }
        }
    }
    if (r.off > 0 && scale != before) {
        const float ratio = __fdiv_rn(before, scale);
        for (int u = tid; u < r.off * d / 16; u += 32 * W) rescale16(r.cache + 16 * u, ratio);
    }
    if (W == 1) __syncwarp();
    // all threads of the run have read the old scale: the maximum brought them together
    if (tid == 0) *r.scale = scale;
}

// G warps take a run together, M vectors of a whole block of tokens to a thread.
template <bool BF16, int G, int M>
__global__ void __launch_bounds__(kThreads, M > 8 ? 2 : (BF16 ? 4 : 3)) cache_write_kernel(CacheWrite p,
                                                                               int tile,
                                                                               int units) {
    __shared__ int32_t at[kMostTile];        // rows of the tile that begin a run
    __shared__ int32_t length[kMostTile];
    __shared__ uint32_t shared[2][kWarps];
    __shared__ int begins;
    const int t0 = blockIdx.x * tile, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int size = 1 << p.block_log2;
    const int vecs_log2 = 31 - __clz(p.d / (BF16 ? 8 : 4));
    const int64_t pool = (int64_t)p.num_blocks << p.block_log2;
    if (w == 0) {
        int n = 0;
        for (int base = 0; base < tile; base += 32) {
            const int i = base + lane, t = t0 + i;
            bool begin = false;
            if (i < tile && t < p.T) {
                const int32_t s = p.slots[t];
                const int32_t ahead = t == 0 ? -1 : p.slots[t - 1];
                begin = s >= 0 && s < pool && ((s & (size - 1)) == 0 || ahead != s - 1);
            }
            const uint32_t all = __ballot_sync(0xffffffffu, begin);
            if (begin) at[n + __popc(all & ((1u << lane) - 1))] = t;
            n += __popc(all);
        }
        if (lane == 0) begins = n;
    }
    __syncthreads();
    const int n = begins;
    if (n == 0) return;
    for (int i = w; i < n; i += kWarps) {
        const int32_t s = p.slots[at[i]];
        const int len = run_length(p.slots, p.T, at[i], s, size - (s & (size - 1)), lane);
        if (lane == 0) length[i] = len;
    }
    __syncthreads();
    // runs that one warp holds, run by run and head by head
    const int first = blockIdx.y * units;
    const int mine = 2 * p.heads - first < units ? 2 * p.heads - first : units;
    for (int i = w; i < n * mine; i += kWarps) {
        const int k = i / mine, len = length[k];
        if (len << vecs_log2 > kShort) continue;
        const Run r = run_of<BF16>(p, first + i - k * mine, at[k], len, p.slots[at[k]]);
        uint4 raw[kShort / 32];
        float before;
        load_run<1>(r, vecs_log2, lane, raw, &before);
        finish_run<BF16, 1>(r, p.d, vecs_log2, lane, raw, before, nullptr, 0);
    }
    if (G == 1) return;
    // the longer ones, G warps to each
    const int group = w / G, tid = threadIdx.x - group * 32 * G;
    int turn = 0;
    for (int i = group; i < n * mine; i += kWarps / G) {
        const int k = i / mine, len = length[k];
        if (len << vecs_log2 <= kShort) continue;
        const Run r = run_of<BF16>(p, first + i - k * mine, at[k], len, p.slots[at[k]]);
        uint4 raw[M];
        float before;
        load_run<G>(r, vecs_log2, tid, raw, &before);
        finish_run<BF16, G>(r, p.d, vecs_log2, tid, raw, before, shared[turn] + group * G,
                            1 + group);
        turn ^= 1;
    }
}

template <bool BF16>
cudaError_t launch_typed(const CacheWrite& p, cudaStream_t stream) {
    // few rows: tiles as large as leave one wave of blocks, each of which has to find its runs
    // before it loads anything.  Against tiles of 8: 3,602 rows of 5 prompts, 3 heads of 64, fp32
    // 9.0 -> 4.0 us, a prompt of 4,096, 8 heads of 128, bf16 10.6 -> 7.4 us; 256, 1,024 and 2,048
    // single tokens of those heads 6.3, 14.8 and 26.7 against 6.4, 16.0 and 29.5 us.
    int tile = p.T <= kFewRows ? 8 : kMostTile;
    while (tile < kMostTile && (int64_t)((p.T + tile - 1) / tile) * 2 * p.heads > kWave) tile *= 2;
    const int tiles = (p.T + tile - 1) / tile;
    // heads of k and v are dealt to as many blocks as keep the SMs busy
    int parts = (kBlocks + tiles - 1) / tiles;
    if (parts > 2 * p.heads) parts = 2 * p.heads;
    const int units = (2 * p.heads + parts - 1) / parts;
    const dim3 grid(tiles, (2 * p.heads + units - 1) / units);
    const int warps = (p.d << p.block_log2) / (BF16 ? 8 : 4) / kShort;   // a block of tokens fills
    auto kernel = warps <= 1   ? cache_write_kernel<BF16, 1, 8>
                  : warps <= 2 ? cache_write_kernel<BF16, 2, 8>
                  : warps <= 4 ? cache_write_kernel<BF16, 4, 8>
                  : warps <= 8 ? cache_write_kernel<BF16, 8, 8>
                               : cache_write_kernel<BF16, 8, BF16 ? 8 : 16>;
    kernel<<<grid, kThreads, 0, stream>>>(p, tile, units);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const CacheWrite& p, int dtype, cudaStream_t stream) {
    return dtype == 0 ? launch_typed<false>(p, stream) : launch_typed<true>(p, stream);
}

}  // namespace kda
