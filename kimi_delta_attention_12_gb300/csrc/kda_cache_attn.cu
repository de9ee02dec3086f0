// kda_cache_attn.cu -- softmax attention over the paged 8-bit cache (kda_cache_attention in
// include/kda.h).
//
// Few rows meet many keys: a decode step reads every cached byte once, so HBM bounds it.  The
// rows of one key and value head (its query heads times the new tokens) are tiles of 8 NT
// columns, and the products stand with the cached tokens as the tensor core's 16 rows:
//
//     S^T = K Q^T        [16 tokens x 8 NT]      A = K, B = Q^T
//     O^T += V^T P^T     [d x 8 NT]              A = V^T, B = P^T
//
// so that eight query rows fill an instruction.  The channels of a product may come in any
// order as long as both sides agree, and the order taken makes every lane's part of a K row 16
// neighbouring bytes: keys and values go from HBM into the registers they are multiplied
// from, no shared memory between.  e4m3 numbers become fp16 exactly; q is scaled by a power of two
// per row (its exponent range is wider than fp16's), for fp32 split into two fp16 halves, and so are
// the weights P.  A row's largest channel comes to [2^14, 2^15), the top of fp16's range: bf16 channels
// are exact down to 2^-31 of it, fp32 ones hold 22 bits down to 2^-17 of it and are off by 2^-39 of it
// below (at [1, 2) a channel 2^-12 of the largest had 13 bits); products with e4m3's 448 at most stay
// far inside fp32.  P^T needs the 8 x 8 transposes of S^T's tiles, one instruction each (movmatrix).
//
// The value scale of a block goes into the exponent: with p' = 2^(s - m + 15) v_scale, m the
// running maximum of s + log2 v_scale, P' is at most 2^15 whatever the scales, and the sum of
// weights takes p' / v_scale.  The 2^15 is for fp16's range: weights down to 2^-29 of the largest
// keep all their bits, and nothing above 2^-40 is lost, however many keys share it.  For bf16 m may
// stay up to 4 below the maximum, at 2^11 instead: a unit whose scores do not pass that, which each
// lane sees for its own, needs no maxima across lanes and no rescaling (256 requests of 4,000 tokens,
// 32 heads over 8, d = 64: 237 -> 214 us; fp32, which keeps the range, 257 -> 235).
//
// Work is cut by tokens, not by requests: all (request, head, row tile) items in a row, each
// ceil(tokens / 64) units, and every block takes the same stretch of units.  An item that lies
// across blocks leaves partial sums, which a second kernel joins.  The 4 warps of a block take
// 16 tokens of a unit each, with sums of their own that meet at the item's end.  A warp has the
// tokens of two units on their way, 8 KB; 12 warps an SM keep HBM busy (d = 128).  128 requests over
// 1.1 M cached tokens, 32 heads over 8, d = 128, bf16: 380 us, 6.4 TB/s, 94 % of the measured copy.
// Prompts in fp32 or of d = 32, which the tensor-core form does not take, come here too, 16 rows a
// tile: 6 requests of 824 new tokens, 15 heads over 3, d = 64, fp32 31 us (35 when each channel of
// the warps' sums was added up for itself; tiles of 32 rows, which spill, took 8 more; 64 rows an
// item, 16 for each warp over all its tokens, 39: four times the partial sums).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kda_cache.h"
#include "kda_e4m3.cuh"
#include "kda_follow.cuh"
#include "kda_seqlens.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kJoinThreads = 256;
constexpr float kNone = -INFINITY;
// In powers of two: how far a weight may pass its reference, and what the reference stands for.
__host__ __device__ constexpr float slack_of(bool F32) { return F32 ? 0.0f : 4.0f; }
__host__ __device__ constexpr float raise_of(bool F32) { return 15.0f - slack_of(F32); }
// From where on prompts go to the tensor cores: rows of the longest request, rows of all heads, and
// those times the tokens that the table can hold.  32 heads over 8, d = 128, one request, us, this
// kernel against that one: 128 / 256 new tokens of 1K 27 against 36 / 38 against 37; 32 / 64 of 8K
// 37 against 43 / 56 against 52; 16 / 32 of 32K 61 against 72 / 99 against 77; 16 heads over 1,
// d = 64: 64 of 8K 26 against 35, 32 of 32K 40 against 47.
constexpr int64_t kManyRows = 64, kManyHeadRows = 1024, kManyWork = (int64_t)1 << 24;
constexpr int kRounds = 32;          // of a warp in a cluster

// Blocks that an SM holds at once, by what a tile needs in registers.  More warps, a few registers
// spilled, beat fewer: single tokens as above, d = 64 with 4 instead of 3 blocks 214 -> 187 us,
// d = 32 with 5 instead of 3 175 -> 140 us, 16 rows there with 4 instead of 3 197 -> 175 us; fp32
// prompts at d = 64 with 3 instead of 2 38.1 -> 35.4 us.
__host__ __device__ constexpr int blocks_per_sm(int NT, int D) {
    return (D == 32 ? 6 : D == 64 ? 5 : 4) - NT;
}

struct Item {
    int request, head, tile;
    int64_t begin;            // where its units begin among all
    int units;
    int tokens, fresh;        // cached, and new ones among them
    int64_t row0;             // of the packed q
};

struct Span {
    int64_t row0;
    int tokens, fresh, tiles, units;
    int64_t all;              // units of the request
};

// UNIT: tokens of a unit, 16 for each warp.
template <int UNIT>
__device__ __forceinline__ Span span_of(const CacheAttention& p, int i, int R) {
    Span s;
    int64_t bos, eos;
    if (p.cu) {
        clamped_seq(p.cu, i, p.N, p.T, bos, eos);
    } else {
        bos = i;
        eos = i + 1;
    }
    // whole units of tokens stay within 32 bits
    const int64_t table = (int64_t)p.width << p.block_log2;
    const int64_t most = table < 0x7fff0000 ? table : 0x7fff0000;
    const int64_t c = p.context[i];
    s.row0 = bos;
    s.fresh = (int)(eos - bos);
    s.tokens = (int)(c < 0 ? 0 : (c < most ? c : most));
    const int64_t rows = (int64_t)s.fresh * p.group;
    s.tiles = rows < p.many_rows ? (int)((rows + R - 1) / R) : 0;
    s.units = s.tokens > 0 ? (int)(((int64_t)s.tokens + UNIT - 1) / UNIT) : 1;
    s.all = (int64_t)s.tiles * p.heads * s.units;
    return s;
}

// a / b, both not negative; 64-bit quotients only where they must be.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// What each block takes: the units begin .. end - 1 of all, and the request that unit `begin`
// belongs to.  All threads of the block; every thread gets the result.
struct Stretch {
    int64_t begin, end, per, first;     // first: where the request's units begin
    int request;
};

template <int THREADS, int UNIT = 16 * kWarps>
__device__ __forceinline__ Stretch stretch_of(const CacheAttention& p, int R, int block,
                                              int blocks) {
    __shared__ int64_t sums[THREADS / 32 + 1];
    __shared__ int64_t found_first;
    __shared__ int found;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int k = (p.N + THREADS - 1) / THREADS;      // requests of a thread, neighbours
    const int i0 = threadIdx.x * k, i1 = i0 + k < p.N ? i0 + k : p.N;
    int64_t mine = 0;
    for (int i = i0; i < i1; ++i) mine += span_of<UNIT>(p, i, R).all;
    int64_t x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sums[w] = x;
    if (threadIdx.x == 0) found = -1;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        before += i < w ? sums[i] : 0;
        total += sums[i];
    }
    Stretch s;
    s.per = quotient(total + blocks - 1, blocks);
    if (s.per < 1) s.per = 1;
    s.begin = s.per * block;
    s.end = s.begin + s.per < total ? s.begin + s.per : total;
    int64_t at = before + x - mine;
    if (s.begin < total && at <= s.begin && s.begin < at + mine) {
        for (int i = i0; i < i1; ++i) {
            const int64_t all = span_of<UNIT>(p, i, R).all;
            if (s.begin < at + all) {
                found = i;
                found_first = at;
                break;
            }
            at += all;
        }
    }
    __syncthreads();
    s.request = found;
    s.first = found_first;
    return s;
}

// The item of unit `at`, from request i on, whose units begin at `first`.
__device__ __forceinline__ Item item_at(const CacheAttention& p, int R, int64_t at, int& i,
                                        int64_t& first) {
    constexpr int UNIT = 16 * kWarps;
    Span s = span_of<UNIT>(p, i, R);
    while (at >= first + s.all && i + 1 < p.N) {
        first += s.all;
        s = span_of<UNIT>(p, ++i, R);
    }
    Item t;
    const int64_t n = quotient(at - first, s.units);
    t.request = i;
    t.head = (int)quotient(n, s.tiles);
    // first, last, second, last but one, ...: under a causal mask a tile and its neighbour together
    // have the same work wherever they stand
    const int k = (int)(n - (int64_t)t.head * s.tiles);
    t.tile = k & 1 ? s.tiles - 1 - (k >> 1) : k >> 1;
    t.begin = first + n * s.units;
    t.units = s.units;
    t.tokens = s.tokens;
    t.fresh = s.fresh;
    t.row0 = s.row0;
    return t;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What is left of lo and hi beside the fp16 pair h.
__device__ __forceinline__ uint32_t rest_of(float lo, float hi, uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return half2_of(lo - f.x, hi - f.y);
}

__device__ __forceinline__ float exp2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The 16 tokens that a warp multiplies at once, as they lie in the cache.
template <int D>
struct Tokens {
    static constexpr int kWords = D >= 64 ? D / 16 : 2;    // of a K row in a lane
    static constexpr int vWords = D / 32;                  // of a V row in a lane
    uint32_t k[2][kWords];
    uint32_t v[4][vWords];
};

// The first channel of word s in a lane's part of a K row; c: the lane's place among four.
template <int D>
__device__ __forceinline__ int k_channel(int s, int c) {
    return D >= 64 ? (s >> 2) * 64 + 16 * c + 4 * (s & 3) : 8 * c + 4 * s;
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t* to, const uint8_t* from) {
    if (N == 4) {
        const uint4 x = __ldcs(reinterpret_cast<const uint4*>(from));
        to[0] = x.x; to[1] = x.y; to[2] = x.z; to[3] = x.w;
    } else if (N == 2) {
        const uint2 x = __ldcs(reinterpret_cast<const uint2*>(from));
        to[0] = x.x; to[1] = x.y;
    } else {
        to[0] = __ldcs(reinterpret_cast<const uint32_t*>(from));
    }
}

template <int D>
__device__ __forceinline__ void load_tokens(const CacheAttention& p, Tokens<D>& x, int head,
                                            int block, int base, int limit, int lane) {
    const int g = lane >> 2, c = lane & 3;
    const bool there = block >= 0 && block < p.num_blocks && base < limit;
    const int64_t tile = ((int64_t)block * p.heads + head) << p.block_log2;
    const int place = base & ((1 << p.block_log2) - 1);
    const uint8_t* k = p.k_cache + (tile + place) * D;
    const uint8_t* v = p.v_cache + (tile + place) * D;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int t = g + 8 * r;
        const bool in = there && base + t < limit;
        if (D >= 64) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                if (in) {
                    load_words<4>(&x.k[r][4 * j], k + t * D + 64 * j + 16 * c);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x.k[r][4 * j + i] = 0;
                }
            }
        } else if (in) {
            load_words<2>(&x.k[r][0], k + t * D + 8 * c);
        } else {
            x.k[r][0] = x.k[r][1] = 0;
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int t = 2 * c + (r & 1) + 8 * (r >> 1);
        if (there && base + t < limit) {
            load_words<D / 32>(&x.v[r][0], v + t * D + g * (D / 8));
        } else {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) x.v[r][i] = 0;
        }
    }
}

// The warps' sums in shared memory: [WARPS][R] rows of sum_stride(D), then their references and
// weights [WARPS][R] each.  Column 2 c + n of an 8-column tile has place 4 n + c there: with the
// rows' 4 floats of padding a half-warp's pairs lie in different banks, or two to a bank.
__host__ __device__ constexpr int sum_stride(int D) { return D + 4; }
__host__ __device__ constexpr int sums_of(int D, int R, int warps) {
    return warps * R * (sum_stride(D) + 2);
}
__device__ __forceinline__ int sum_place(int n) { return (n & ~7) + 4 * (n & 1) + ((n & 7) >> 1); }

// Units unit0 .. unit0 + units - 1 of an item by WARPS warps: every warp's sums into `sums`.
template <int D, int NT, bool F32, int WARPS>
__device__ __forceinline__ void attend(const CacheAttention& p, const Item& it, int unit0,
                                       int units, float* sums) {
    constexpr int R = 8 * NT, kSteps = D / 16, Q = F32 ? 2 : 1, UNIT = 16 * WARPS;
    constexpr int S = sum_stride(D);
    float* sums_m = sums + WARPS * R * S;
    float* sums_l = sums_m + WARPS * R;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int rows = it.fresh * p.group - it.tile * R;      // of this tile, may be above R
    const int hidden = it.tokens - it.fresh + 1;            // keys that new token 0 sees
    const int last = rows < R ? rows : R;
    const int low = hidden + it.tile * R / p.group;                  // what the tile's first row
    const int high = hidden + (it.tile * R + last - 1) / p.group;    // and its last row see
    if (R == 16) {                       // a prompt's tiles end before its tokens do
        const int past = high > 0 ? (high - 1) / UNIT + 1 - unit0 : 0;
        if (units > past) units = past;
    }
    // ---- the first tokens on their way
    const int32_t* table = p.table + (int64_t)it.request * p.width;
    int ids = -1;                        // of the blocks of 32 units, one in each lane
    float k_scale = 0.0f, v_log = 0.0f, v_inverse = 1.0f;
    auto look_up = [&](int u) {
        const int base = (unit0 + u + lane) * UNIT + 16 * w;
        ids = u + lane < units && base < high ? table[base >> p.block_log2] : -1;
        k_scale = 0.0f;
        v_log = 0.0f;
        v_inverse = 1.0f;
        if (ids >= 0 && ids < p.num_blocks) {
            k_scale = p.k_scale[(int64_t)ids * p.heads + it.head];
            const float v_scale = p.v_scale[(int64_t)ids * p.heads + it.head];
            v_log = __log2f(v_scale);
            v_inverse = __frcp_rn(v_scale);
        }
    };
    int u0 = 0, n = units < 32 ? units : 32;     // units of which `ids` holds the blocks
    Tokens<D> x, y;
    auto load = [&](Tokens<D>& to, int u) {
        load_tokens<D>(p, to, it.head, __shfl_sync(0xffffffffu, ids, u & 31),
                       (unit0 + u0 + u) * UNIT + 16 * w, u < n ? high : 0, lane);
    };
    look_up(0);
    load(x, 0);
    load(y, 1);
    // ---- q of this lane's column, its largest channel scaled to [2^14, 2^15), in fp16
    uint32_t q[Q][NT][kSteps][2];
    float factor[NT][2];                 // of a score, for the columns 2 c and 2 c + 1
    int limit[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int own = 8 * t + g, flat = it.tile * R + own, j = flat / p.group;
        float v[kSteps][4], top = 0.0f;
        const int64_t base = (it.row0 + j) * p.q_stride +
                             (int64_t)(it.head * p.group + flat - j * p.group) * D;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int d = k_channel<D>(i, c);
            if (own >= rows) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = 0.0f;
            } else if (F32) {
                const float4 f = *reinterpret_cast<const float4*>(
                    static_cast<const float*>(p.q) + base + d);
                v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
            } else {
                const uint2 f = *reinterpret_cast<const uint2*>(
                    static_cast<const __nv_bfloat16*>(p.q) + base + d);
                v[i][0] = __uint_as_float(f.x << 16);
                v[i][1] = __uint_as_float(f.x & 0xffff0000u);
                v[i][2] = __uint_as_float(f.y << 16);
                v[i][3] = __uint_as_float(f.y & 0xffff0000u);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(v[i][e]));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = __float_as_int(top) >> 23;
        e = e < 15 ? 15 : (e > 254 ? 254 : e);
        const float down = __int_as_float((268 - e) << 23), up = __int_as_float((e - 14) << 23);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float lo = v[i][2 * b] * down, hi = v[i][2 * b + 1] * down;
                q[0][t][i][b] = half2_of(lo, hi);
                if (F32) q[Q - 1][t][i][b] = rest_of(lo, hi, q[0][t][i][b]);
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int col = 2 * c + b;
            factor[t][b] = __shfl_sync(0xffffffffu, up, 4 * col) *
                           (p.scale * 1.44269504088896340736f);
            const int nb = 8 * t + col, fb = it.tile * R + nb;
            limit[t][b] = nb < rows ? hidden + fb / p.group : 0x7fffffff;
        }
    }
    // ---- this warp's part of the units
    float o[NT][kSteps][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t][0] = m[t][1] = kNone;
        l[t][0] = l[t][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.0f;
        }
    }
    auto multiply = [&](const Tokens<D>& x, int u, float ks, float lv, float iv, bool there) {
        const int base = (unit0 + u) * UNIT + 16 * w;
        if (base >= high || !there) return;
        float sc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const uint32_t a0 = half2_of_e4m3(x.k[0][i]), a1 = half2_of_e4m3(x.k[1][i]);
            const uint32_t a2 = half2_of_e4m3_high(x.k[0][i]);
            const uint32_t a3 = half2_of_e4m3_high(x.k[1][i]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int h = 0; h < Q; ++h) {
                    mma(sc[t], a0, a1, a2, a3, q[h][t][i][0], q[h][t][i][1]);
                }
            }
        }
        const bool partly = base + 16 > low;
        uint32_t b[Q][NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float f = factor[t][n] * ks;
                float s0 = fmaf(sc[t][n], f, lv), s1 = fmaf(sc[t][n + 2], f, lv);
                if (partly) {
                    s0 = base + g < limit[t][n] ? s0 : kNone;
                    s1 = base + g + 8 < limit[t][n] ? s1 : kNone;
                }
                sc[t][n] = s0;
                sc[t][n + 2] = s1;
            }
        }
        bool more = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                more |= fmaxf(sc[t][n], sc[t][n + 2]) > m[t][n] + slack_of(F32);
            }
        }
        if (__any_sync(0xffffffffu, more)) {
            float up[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float x = fmaxf(sc[t][n], sc[t][n + 2]);
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    up[t][n] = fmaxf(m[t][n], x);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float less[2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    less[n] = up[t][n] > m[t][n] ? exp2_of(m[t][n] - up[t][n]) : 1.0f;
                    m[t][n] = up[t][n];
                    l[t][n] *= less[n];
                }
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    o[t][i][0] *= less[0];
                    o[t][i][1] *= less[1];
                    o[t][i][2] *= less[0];
                    o[t][i][3] *= less[1];
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float e[4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float top = (m[t][n] == kNone ? 0.0f : m[t][n]) - raise_of(F32);
                e[n] = exp2_of(sc[t][n] - top);
                e[n + 2] = exp2_of(sc[t][n + 2] - top);
                l[t][n] = fmaf(e[n] + e[n + 2], iv, l[t][n]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t pair = half2_of(e[2 * h], e[2 * h + 1]);
                b[0][t][h] = transposed(pair);
                if (F32) {
                    b[Q - 1][t][h] = transposed(rest_of(e[2 * h], e[2 * h + 1], pair));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            // channels 2 i and 2 i + 1 of this lane's D / 8, of four tokens
            uint32_t pair[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                pair[h] = __byte_perm(x.v[2 * h][i / 2], x.v[2 * h + 1][i / 2],
                                      i & 1 ? 0x7362 : 0x5140);
            }
            const uint32_t a0 = half2_of_e4m3(pair[0]), a1 = half2_of_e4m3_high(pair[0]);
            const uint32_t a2 = half2_of_e4m3(pair[1]), a3 = half2_of_e4m3_high(pair[1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int h = 0; h < Q; ++h) mma(o[t][i], a0, a1, a2, a3, b[h][t][0], b[h][t][1]);
            }
        }
    };
    auto take = [&](const Tokens<D>& from, int u) {
        const int id = __shfl_sync(0xffffffffu, ids, u);
        const float ks = __shfl_sync(0xffffffffu, k_scale, u);
        const float lv = __shfl_sync(0xffffffffu, v_log, u);
        const float iv = __shfl_sync(0xffffffffu, v_inverse, u);
        multiply(from, u0 + u, ks, lv, iv, id >= 0 && id < p.num_blocks);
    };
    while (u0 < units) {
        for (int u = 0; u < n; u += 2) {
            take(x, u);
            load(x, u + 2);
            if (u + 1 < n) take(y, u + 1);
            load(y, u + 3);
        }
        u0 += 32;
        if (u0 >= units) break;
        n = units - u0 < 32 ? units - u0 : 32;
        look_up(u0);
        load(x, 0);
        load(y, 1);
    }
    // ---- the warps' sums, to where they meet
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                l[t][n] += __shfl_xor_sync(0xffffffffu, l[t][n], d);
            }
            const int col = 8 * t + 4 * n + c;
            if (g == 0) {
                sums_m[w * R + col] = m[t][n];
                sums_l[w * R + col] = l[t][n];
            }
            float* to = sums + (w * R + col) * S + g * (D / 8);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                *reinterpret_cast<float2*>(to + 2 * i) = make_float2(o[t][i][n], o[t][i][n + 2]);
            }
        }
    }
}

// Channels d .. d + 3 of row n from the warps' sums, with the reference and weight of all of them.
template <int D, int R, int WARPS>
__device__ __forceinline__ float4 meet(const float* sums, int n, int d, float& weight, float& top) {
    constexpr int S = sum_stride(D);
    const int place = sum_place(n);
    const float* sums_m = sums + WARPS * R * S + place;
    const float* sums_l = sums_m + WARPS * R;
    top = kNone;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) top = fmaxf(top, sums_m[k * R]);
    const float ref = top == kNone ? 0.0f : top;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    weight = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
        const float f = exp2_of(sums_m[k * R] - ref);
        const float4 x = *reinterpret_cast<const float4*>(sums + (k * R + place) * S + d);
        y.x = fmaf(f, x.x, y.x);
        y.y = fmaf(f, x.y, y.y);
        y.z = fmaf(f, x.z, y.z);
        y.w = fmaf(f, x.w, y.w);
        weight = fmaf(f, sums_l[k * R], weight);
    }
    return y;
}

// Where row n of an item's tile goes in o.
__device__ __forceinline__ int64_t place_of(const CacheAttention& p, const Item& it, int R, int n,
                                            int D) {
    const int flat = it.tile * R + n, j = flat / p.group;
    return ((it.row0 + j) * (p.heads * p.group) + it.head * p.group + flat - j * p.group) * D;
}

// Four neighbouring channels of the result: the sums over `weight`, 0 where nothing was seen (whose
// sums are weights of 0 times values that may be NaN).
template <bool F32>
__device__ __forceinline__ void store4(void* o, int64_t to, const float4& sums, float weight) {
    const bool none = weight == 0.0f;
    const float by = none ? 0.0f : 1.0f / weight;
    const float4 y = make_float4(none ? 0.0f : sums.x * by, none ? 0.0f : sums.y * by,
                                 none ? 0.0f : sums.z * by, none ? 0.0f : sums.w * by);
    if (F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(o) + to) = y;
    } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(y.z, y.w);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(o) + to) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                       *reinterpret_cast<const uint32_t*>(&hi));
    }
}

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(NT, D)) cache_attention_kernel(
    CacheAttention p) {
    constexpr int R = 8 * NT;
    extern __shared__ __align__(16) float sums[];
    let_follow();
    if (p.clears && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    const Stretch s = stretch_of<kThreads>(p, R, blockIdx.x, gridDim.x);
    int request = s.request;
    int64_t first = s.first;
    for (int64_t at = s.begin; request >= 0 && at < s.end;) {
        const Item it = item_at(p, R, at, request, first);
        const int unit0 = (int)(at - it.begin);
        const int units = (int)(s.end - at < it.units - unit0 ? s.end - at : it.units - unit0);
        attend<D, NT, F32, kWarps>(p, it, unit0, units, sums);
        __syncthreads();
        const int rows = it.fresh * p.group - it.tile * R, valid = rows < R ? rows : R;
        const bool whole = unit0 == 0 && units == it.units;
        float* part = p.partial + (int64_t)(blockIdx.x * 2 + (at != s.begin)) * R * (D + 2);
        for (int i = 4 * threadIdx.x; i < valid * D; i += 4 * kThreads) {
            const int n = i / D, d = i - n * D;
            float weight, top;
            const float4 y = meet<D, R, kWarps>(sums, n, d, weight, top);
            if (whole) {
                store4<F32>(p.o, place_of(p, it, R, n, D) + d, y, weight);
            } else {
                *reinterpret_cast<float4*>(part + i) = y;
                if (d == 0) {
                    part[R * D + n] = top;
                    part[R * D + R + n] = weight;
                }
            }
        }
        __syncthreads();
        at += units;
    }
    // behind the prompts' kernel, whose sums this one does not need: its end follows that one's
    if (blockIdx.x == gridDim.x - 1) wait_before();
}

// Few requests and heads: a cluster of blocks for each, which share its tokens and join their sums
// through one another's shared memory, all in one launch.
__host__ __device__ constexpr int cluster_warps(int NT) { return NT == 1 ? 8 : 4; }

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(32 * cluster_warps(NT), 1) cache_attention_cluster_kernel(
    CacheAttention p) {
    namespace cg = cooperative_groups;
    constexpr int R = 8 * NT, W = cluster_warps(NT), kAll = 32 * W;
    // the warps' sums, then this block's: [R][D], m, l [R]
    extern __shared__ __align__(16) float sums[];
    float* block_o = sums + sums_of(D, R, W);
    float* block_m = block_o + R * D;
    float* block_l = block_m + R;
    if (p.clears && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int item = blockIdx.x / blocks;
    Item it;
    it.request = item / p.heads;
    it.head = item - it.request * p.heads;
    const Span s = span_of<16 * W>(p, it.request, R);
    it.units = s.units;
    it.tokens = s.tokens;
    it.fresh = s.fresh;
    it.row0 = s.row0;
    const int per = (s.units + blocks - 1) / blocks;
    const int unit0 = rank * per < s.units ? rank * per : s.units;
    const int units = s.units - unit0 < per ? s.units - unit0 : per;
    for (it.tile = 0; it.tile < s.tiles; ++it.tile) {
        attend<D, NT, F32, W>(p, it, unit0, units, sums);
        __syncthreads();
        const int rows = it.fresh * p.group - it.tile * R, valid = rows < R ? rows : R;
        for (int i = 4 * threadIdx.x; i < valid * D; i += 4 * kAll) {
            const int n = i / D, d = i - n * D;
            float weight, top;
            *reinterpret_cast<float4*>(block_o + i) = meet<D, R, W>(sums, n, d, weight, top);
            if (d == 0) {
                block_m[n] = top;
                block_l[n] = weight;
            }
        }
        cluster.sync();
        for (int i = rank * kAll + threadIdx.x; i < valid * D / 4; i += blocks * kAll) {
            const int n = 4 * i / D;
            float top = kNone, all = 0.0f;
            for (int k = 0; k < blocks; ++k) {
                top = fmaxf(top, cluster.map_shared_rank(block_m, k)[n]);
            }
            const float ref = top == kNone ? 0.0f : top;
            float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int k = 0; k < blocks; ++k) {
                const float f = exp2_of(cluster.map_shared_rank(block_m, k)[n] - ref);
                const float4 x =
                    *reinterpret_cast<const float4*>(cluster.map_shared_rank(block_o, k) + 4 * i);
                all = fmaf(f, cluster.map_shared_rank(block_l, k)[n], all);
                y.x = fmaf(f, x.x, y.x);
                y.y = fmaf(f, x.y, y.y);
                y.z = fmaf(f, x.z, y.z);
                y.w = fmaf(f, x.w, y.w);
            }
            store4<F32>(p.o, place_of(p, it, R, n, D) + 4 * i - n * D, y, all);
        }
        cluster.sync();                      // the others may still read this block's sums
    }
}

// Joins the parts of the item that ends among block blockIdx.x's units and began before them.
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kJoinThreads) cache_attention_join_kernel(CacheAttention p) {
    constexpr int R = 8 * NT, kStride = R * (D + 2);
    extern __shared__ float weights[];       // [R][blocks of the item]
    __shared__ float total[R];
    __shared__ float4 shares[kJoinThreads];
    const Stretch s = stretch_of<kJoinThreads>(p, R, blockIdx.x, gridDim.x);
    wait_before();
    if (s.request < 0) return;
    int request = s.request;
    int64_t first = s.first;
    const Item it = item_at(p, R, s.begin, request, first);
    if (it.begin == s.begin || it.begin + it.units > s.end) return;
    const int rows = it.fresh * p.group - it.tile * R, valid = rows < R ? rows : R;
    const int b0 = (int)quotient(it.begin, s.per), parts = blockIdx.x - b0 + 1;
    auto part_of = [&](int k) {
        const bool second = k == 0 && it.begin != b0 * s.per;
        return p.partial + (int64_t)((b0 + k) * 2 + second) * kStride;
    };
    const int lane = threadIdx.x & 31;
    for (int n = threadIdx.x >> 5; n < valid; n += kJoinThreads / 32) {
        float top = kNone;
        for (int k = lane; k < parts; k += 32) top = fmaxf(top, part_of(k)[R * D + n]);
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float ref = top == kNone ? 0.0f : top;
        float sum = 0.0f;
        for (int k = lane; k < parts; k += 32) {
            const float* part = part_of(k) + R * D + n;
            const float f = exp2_of(part[0] - ref);
            weights[n * parts + k] = f;
            sum = fmaf(f, part[R], sum);
        }
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) total[n] = sum;
    }
    __syncthreads();
    // four channels to a thread; the threads left over share the parts
    const int outs = valid * D / 4;
    const int sharers = outs >= kJoinThreads ? 1 : kJoinThreads / outs;
    for (int i0 = 0; i0 < outs; i0 += kJoinThreads) {
        const int share = i0 + kJoinThreads <= outs || sharers == 1 ? 0 : threadIdx.x / outs;
        const int i = i0 + (sharers == 1 ? threadIdx.x : threadIdx.x - share * outs);
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int n = 4 * i / D, d = 4 * i - n * D;
        if (i < outs && share < sharers) {
#pragma unroll 8
            for (int k = share; k < parts; k += sharers) {
                const float f = weights[n * parts + k];
                const float4 x = *reinterpret_cast<const float4*>(part_of(k) + 4 * i);
                y.x = fmaf(f, x.x, y.x);
                y.y = fmaf(f, x.y, y.y);
                y.z = fmaf(f, x.z, y.z);
                y.w = fmaf(f, x.w, y.w);
            }
        }
        if (sharers > 1) {
            shares[threadIdx.x] = y;
            __syncthreads();
            if (share > 0 || i >= outs) return;
            for (int k = 1; k < sharers; ++k) {
                const float4 x = shares[k * outs + i];
                y.x += x.x;
                y.y += x.y;
                y.z += x.z;
                y.w += x.w;
            }
        }
        if (i >= outs) return;
        store4<F32>(p.o, place_of(p, it, R, n, D) + d, y, total[n]);
    }
}

// Blocks of a cluster for each item of the call, 1: none.  Every SM gets a block at most, with
// clusters of 8 every other one (they lie within a group of SMs, and 16 of them did not fit at
// once), and a warp at most kRounds times 16 tokens; beyond, the even stretches over all SMs are
// faster although they take two launches.  8 heads of d = 128, 4 rows each, clusters against
// stretches, us: 1 request of 1K, 8K, 32K, 128K tokens 6.1, 10.4, 24.2, 106 against 11.1, 19.2,
// 26.4, 58.8 (8 a cluster); 4 of 8K, 16K, 32K 15.2, 32.1, 58.9 against 21.5, 34.2, 53.9 (4); 8 of
// 8K 32.0 against 33.7, 9 of 1K 8.1 against 15.9 (2).  Clusters of 16 took 17.0 for 1 of 8K, when
// 8 took 11.4.
int cluster_of(const CacheAttention& p, int sms, int NT) {
    const int64_t items = (int64_t)p.N * p.heads, most = (int64_t)p.width << p.block_log2;
    for (int c = 8; c > 1; c /= 2) {
        const bool fits = items * c <= (c == 8 ? sms / 2 : sms);
        if (fits && most <= (int64_t)kRounds * c * 16 * cluster_warps(NT)) return c;
    }
    return 1;
}

template <int D, int NT, bool F32>
cudaError_t launch_clusters(const CacheAttention& p, int blocks, cudaStream_t stream) {
    auto kernel = cache_attention_cluster_kernel<D, NT, F32>;
    constexpr int R = 8 * NT, W = cluster_warps(NT);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(p.N * p.heads * blocks);
    config.blockDim = dim3(32 * W);
    config.dynamicSmemBytes = (size_t)(sums_of(D, R, W) + R * (D + 2)) * sizeof(float);
    config.stream = stream;
    config.attrs = &attr;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, kernel, p);
}

template <int D, int NT, bool F32>
cudaError_t launch_tiles(const CacheAttention& p, int sms, cudaStream_t stream) {
    constexpr int R = 8 * NT;
    // (rows that fill one tile at most: the work is the tokens alone)
    const int cluster = (int64_t)p.group * p.max_new <= R ? cluster_of(p, sms, NT) : 1;
    if (cluster > 1) {
        if (launch_clusters<D, NT, F32>(p, cluster, stream) == cudaSuccess) return cudaSuccess;
        cudaGetLastError();                  // a device that cannot take them (a part of a GPU)
    }
    const size_t smem = (size_t)sums_of(D, R, kWarps) * sizeof(float);
    const int blocks = sms * blocks_per_sm(NT, D);
    cudaError_t err;
    if (p.many_rows == INT64_MAX) {
        cache_attention_kernel<D, NT, F32><<<blocks, kThreads, smem, stream>>>(p);
        err = cudaGetLastError();
    } else {
        // on SMs that the prompts leave idle or are done with; what joins their parts waits for
        // both (63 single tokens and a prompt of 200 as above 105 -> 86 us)
        err = launch_follower(cache_attention_kernel<D, NT, F32>, dim3(blocks), dim3(kThreads),
                              smem, stream, p);
        if (err == cudaSuccess) err = launch_cache_prompt_join(p, sms, stream);
    }
    if (err != cudaSuccess) return err;
    return launch_follower(cache_attention_join_kernel<D, NT, F32>, dim3(blocks),
                           dim3(kJoinThreads), (size_t)R * blocks * sizeof(float), stream, p);
}

template <int D, bool F32>
cudaError_t launch_dim(const CacheAttention& p, int sms, cudaStream_t stream) {
    // one column tile where the rows of every request fit it, else two: half the reads of K and V.
    // Beside the tensor cores' kernel the other requests' rows count, at their average: 63 single
    // tokens, 200 new ones, 32 heads over 8, d = 128, behind 2,000 each 122 -> 105 us; 64 times 4
    // and 500 behind 4,000, which stay with two, 169 against 213.
    const int64_t rows = p.many_rows == INT64_MAX ? (int64_t)p.group * p.max_new
                         : (int64_t)p.group * (p.T - p.max_new) / (p.N - 1);
    return rows <= 8 ? launch_tiles<D, 1, F32>(p, sms, stream)
                     : launch_tiles<D, 2, F32>(p, sms, stream);
}

template <bool F32>
cudaError_t launch_typed(const CacheAttention& p, int sms, cudaStream_t stream) {
    switch (p.d) {
        case 32: return launch_dim<32, F32>(p, sms, stream);
        case 64: return launch_dim<64, F32>(p, sms, stream);
        default: return launch_dim<128, F32>(p, sms, stream);
    }
}

}  // namespace

bool cache_prompt_used(int32_t heads, int32_t group, int32_t T, int32_t max_new, int32_t d,
                       int dtype) {
    return cache_prompt_takes(d, dtype) && (int64_t)group * max_new >= kManyRows &&
           (int64_t)group * T * heads >= kManyHeadRows;
}

size_t cache_attention_room(int32_t heads, int32_t group, int32_t T, int32_t max_new, int32_t d,
                            int dtype, int sms) {
    const int most = blocks_per_sm(2, d) * 16;       // rows of an SM's tiles
    const size_t room = (size_t)sms * most * 2 * (d + 2) * sizeof(float);
    const size_t prompts = cache_prompt_used(heads, group, T, max_new, d, dtype)
                               ? cache_prompt_room(d, sms) : 0;
    return prompts + room;
}

cudaError_t launch_cache_attention(const CacheAttention& call, int dtype, int sms,
                                   cudaStream_t stream) {
    CacheAttention p = call;
    p.clears = 1;
    p.many_rows = INT64_MAX;
    const double work = (double)p.group * p.T * p.heads * ((int64_t)p.width << p.block_log2);
    if (cache_prompt_used(p.heads, p.group, p.T, p.max_new, p.d, dtype) && work >= kManyWork) {
        p.many_rows = p.N == 1 ? 1 : kManyRows;
        p.prompt_partial = p.partial;
        p.partial += cache_prompt_room(p.d, sms) / sizeof(float);
        const cudaError_t err = launch_cache_prompt(p, sms, stream);
        if (err != cudaSuccess) return err;
        if (p.N == 1) return launch_cache_prompt_join(p, sms, stream);
        p.clears = 0;
    }
    return dtype == 0 ? launch_typed<true>(p, sms, stream) : launch_typed<false>(p, sms, stream);
}

}  // namespace kda
