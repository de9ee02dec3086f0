// kda_rotary.cu -- rotary positions of q and k, forward and backward (kda_rotary in
// include/kda.h): pair (u, w) becomes magnitude (u cos a - w sin a, u sin a + w cos a) with
// a = position * inv_freq.
//
// The angle.  Only its fraction of a turn matters, so the frequency is held as a 64-bit
// fraction F = f / (2 pi) mod 1 and the phase is the wrapping integer product p F: exact to
// 2^-41 of a turn at a position of 2^23, where an fp32 product of the two would have lost
// the angle altogether.  F comes from the 24 mantissa bits of f and the first 64 bits of
// 1 / (2 pi) by one integer product and a shift, no 64-bit floating point.  The upper 32 bits
// of the phase become half turns in [-1, 1) for sincospif.
//
// Bound by HBM: every value is read and written once, three operations each.  A block takes a
// stretch of (token, head) rows, forms the cosines and sines of its few tokens once in shared
// memory (all heads of a token share them) while its first rows are on their way, and turns
// 16-byte vectors: a vector of neighbouring channels, or two that lie rot / 2 apart.  A thread has
// one vector ahead of the one that it stores, and 48 warps an SM do the rest: four ahead took 90
// registers and 723 us where 65,536 rows of 96 + 8 heads, 64 of 128 channels turned, bf16, take 530
// (6.6 TB/s, 98 % of the measured copy).
#include <cuda_bf16.h>

#include "kda_cache.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
// Vectors (or pairs of them) of a block.
constexpr int kLeastUnits = 512, kMostUnits = 4096;
constexpr int kBlocks = 1216;        // that a large call aims at: eight for each of GB300's 152 SMs, which
                                     // hold six at once

// f / (2 pi) as a 64-bit fraction of a turn, whole turns dropped.
__device__ __forceinline__ uint64_t turns_of(float f) {
    // 1 / (2 pi) = 0.28BE60DB 9391054A ... in base 16: the binary digits of 0.159154943...
    constexpr uint64_t kInvTwoPi = 0x28BE60DB9391054Aull;
    const uint32_t bits = __float_as_uint(f);
    const int e = (bits >> 23) & 255;
    const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    // f = m 2^-s: the product m * kInvTwoPi (88 bits) shifted right by s
    const int s = 150 - (e ? e : 1);
    const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
    uint64_t F;
    if (s <= -64) {
        F = 0;
    } else if (s < 0) {
        F = lo << -s;
    } else if (s == 0) {
        F = lo;
    } else if (s < 64) {
        F = (hi << (64 - s)) | (lo >> s);
    } else {
        F = s < 128 ? hi >> (s - 64) : 0;
    }
    return (bits >> 31) ? 0 - F : F;
}

// cos and sin of the angle, times the magnitude.
__device__ __forceinline__ float2 turn(int32_t position, float f, float magnitude, bool inverse) {
    const uint64_t phase = (uint64_t)(int64_t)position * turns_of(f);
    float sn, cs;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
    return make_float2(cs * magnitude, (inverse ? -sn : sn) * magnitude);
}

template <bool BF16>
struct Vec {
    static constexpr int n = BF16 ? 8 : 4;
    uint4 raw;
    __device__ __forceinline__ void get(float* x) const {
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
    __device__ __forceinline__ void put(const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (BF16) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
                w[i] = __float_as_uint(x[i]);
            }
        }
        raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// How a thread gets from one of its units to the next: kThreads units on.
struct Steps {
    int units, turned;       // of a row; of those, the turned ones
    int in_row, tokens, heads;   // kThreads units as rows and a rest, the rows as tokens and a rest
};

// Rows of a call in order: token, then the heads of q, then those of k.  A row is cut into
// `units`: the turned vectors (or pairs of vectors), then the ones that are copied.
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads, 6) rotary_kernel(Rotary p, int rows_per_block,
                                                          const Steps step) {
    using V = Vec<BF16>;
    constexpr int n = V::n, size = BF16 ? 2 : 4;
    extern __shared__ float2 table[];        // [tokens of this block][rot / 2]
    const int heads = p.heads[0] + p.heads[1], half = p.rot / 2;
    const int64_t total = p.T * heads, row0 = (int64_t)blockIdx.x * rows_per_block;
    const int rows = (int)(total - row0 < rows_per_block ? total - row0 : rows_per_block);
    const int64_t t0 = row0 / heads;
    const int head0 = (int)(row0 - t0 * heads);
    const int tokens = (head0 + rows - 1) / heads + 1;

    struct Unit {
        char* to;
        const float2* angles;
        bool turned;
        V a, b;
    };
    // where this thread is
    int in_row = threadIdx.x % step.units, dt = (head0 + threadIdx.x / step.units) / heads;
    int head = head0 + threadIdx.x / step.units - dt * heads, left = rows * step.units - threadIdx.x;
    auto load = [&](Unit& x) {
        if (left > 0) {
            const bool second = head >= p.heads[0];
            const int h = second ? head - p.heads[0] : head;
            x.turned = in_row < step.turned;
            int c;                           // the unit's first channel
            if (x.turned) {
                c = p.first + in_row * n;
                x.angles = table + dt * half + (INTER ? in_row * n / 2 : in_row * n);
            } else {
                c = (in_row - step.turned) * n;
                c += c >= p.first ? p.rot : 0;
            }
            const int64_t col = h * p.d + c, t = t0 + dt;
            const char* from = static_cast<const char*>(second ? p.x[1] : p.x[0]) +
                               (t * (second ? p.stride[1] : p.stride[0]) + col) * size;
            x.to = static_cast<char*>(second ? p.out[1] : p.out[0]) +
                   (t * (second ? p.out_stride[1] : p.out_stride[0]) + col) * size;
            x.a.raw = __ldcs(reinterpret_cast<const uint4*>(from));
            if (!INTER && x.turned) {
                x.b.raw = __ldcs(reinterpret_cast<const uint4*>(from + half * size));
            }
        } else {
            x.to = nullptr;
        }
        left -= kThreads;
        in_row += step.in_row;
        head += step.heads;
        dt += step.tokens;
        if (in_row >= step.units) {
            in_row -= step.units;
            ++head;
        }
        if (head >= heads) {                 // (below 2 heads: step.heads is below heads)
            head -= heads;
            ++dt;
        }
    };
    auto finish = [&](Unit& x) {
        if (x.to == nullptr) return;
        if (x.turned) {
            float u[n], w[n];
            x.a.get(u);
            if (INTER) {
#pragma unroll
                for (int i = 0; i < n / 2; ++i) {
                    const float2 cs = x.angles[i];
                    w[2 * i] = u[2 * i] * cs.x - u[2 * i + 1] * cs.y;
                    w[2 * i + 1] = u[2 * i] * cs.y + u[2 * i + 1] * cs.x;
                }
                x.a.put(w);
            } else {
                x.b.get(w);
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float2 cs = x.angles[i];
                    const float y = u[i] * cs.x - w[i] * cs.y;
                    w[i] = u[i] * cs.y + w[i] * cs.x;
                    u[i] = y;
                }
                x.a.put(u);
                x.b.put(w);
                __stcs(reinterpret_cast<uint4*>(x.to + half * size), x.b.raw);
            }
        }
        __stcs(reinterpret_cast<uint4*>(x.to), x.a.raw);
    };

    // one unit ahead of the one that is stored
    Unit x, y;
    load(x);
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        table[i] = turn(p.positions[t0 + t], p.inv_freq[j], p.magnitude, p.inverse);
    }
    __syncthreads();
    while (x.to != nullptr) {
        load(y);
        finish(x);
        if (y.to == nullptr) break;
        load(x);
        finish(y);
    }
}

template <bool BF16>
cudaError_t launch_typed(const Rotary& p, cudaStream_t stream) {
    constexpr int n = BF16 ? 8 : 4;
    // in place the channels that are not turned need no pass
    bool copy = false;
    for (int i = 0; i < 2; ++i) copy |= p.heads[i] > 0 && p.out[i] != p.x[i];
    const int turned = p.rot / n / (p.interleaved ? 1 : 2);
    const int units = turned + (copy ? (p.d - p.rot) / n : 0);
    const int64_t heads = p.heads[0] + p.heads[1], total = p.T * heads;
    // long stretches keep loads ahead of the stores, short ones keep all SMs busy
    int64_t most_units = total * units / kBlocks;
    most_units = most_units < kLeastUnits ? kLeastUnits
                                          : (most_units > kMostUnits ? kMostUnits : most_units);
    int rows = (int)((most_units + units - 1) / units);
    const int64_t half = p.rot / 2;
    // the table of a block's tokens stays within 32 KB
    const int64_t most = (32768 / (half * 8) - 1) * heads;
    if (rows > most) rows = most < 1 ? 1 : (int)most;
    const int64_t tokens = (rows + heads - 2) / heads + 1;
    const int64_t blocks = (total + rows - 1) / rows;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    Steps step;
    step.units = units;
    step.turned = turned;
    step.in_row = kThreads % units;
    step.tokens = (int)(kThreads / units / heads);
    step.heads = (int)(kThreads / units % heads);
    const size_t smem = (size_t)(tokens * half) * sizeof(float2);
    auto kernel = p.interleaved ? rotary_kernel<BF16, true> : rotary_kernel<BF16, false>;
    kernel<<<(unsigned)blocks, kThreads, smem, stream>>>(p, rows, step);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const Rotary& p, int dtype, cudaStream_t stream) {
    return dtype == 0 ? launch_typed<false>(p, stream) : launch_typed<true>(p, stream);
}

}  // namespace kda
