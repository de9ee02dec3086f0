// kda_cache_prompt_sm103.cu -- softmax attention over the paged 8-bit cache for prompts, on the
// fifth-generation tensor cores (kda_cache_attention in include/kda.h; bf16, d = 64 or 128).
//
// Many rows meet every key: 4 pairs d operations against a few bytes, so the tensor core bounds
// it, and next to it the exponentials (one for every 4 d operations).  A CTA takes 256 rows of one
// key and value head (its query heads times neighbouring new tokens) as two tiles of 128, and
// walks the cached tokens 128 at a time:
//
//     S = Q K^T    128 x 128 a tile, Q and K in shared memory, S in TMEM
//     P = 2^(S f - m)    one thread a row, written back over S as fp16 pairs
//     O += P V     P from TMEM, V from shared memory, O in TMEM
//
// The tiles take turns: while one's softmax runs, the tensor core works for the other.  Roles:
// warps 0-7 a row each (softmax, the output), warps 8-11 read e4m3 tiles of the cache and write
// them as fp16 (exact) in the operands' layout, warp 12 issues the products.
//
// fp16, not bf16: e4m3 numbers and, scaled to [1, 2) by a power of two per row, bf16 queries are
// fp16 numbers, and P keeps 11 bits.  Scales of key blocks go into the exponent's factor, those
// of value blocks into its offset, as in the kernel for few rows: p' = 2^(s - m + 7) v_scale with
// m at most 8 below the running maximum of s + log2 v_scale.  That slack is what spares most tiles
// the rescaling of O: it is done where the maximum has grown by more, and P stays below 2^15.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kda_cache.h"
#include "kda_e4m3.cuh"
#include "kda_seqlens.cuh"
#include "sm103_ptx.cuh"

namespace kda {
namespace {

using namespace sm103;

constexpr int kRows = 128;               // of a tile
constexpr int kTokens = 128;             // of a step
constexpr int kSoftWarps = 8, kFillWarps = 4;
constexpr int kIssueWarp = kSoftWarps + kFillWarps;
constexpr int kThreads = 32 * (kIssueWarp + 1);
constexpr float kNone = -INFINITY;
constexpr float kSlack = 8.0f, kRaise = 7.0f;
constexpr uint32_t kHalf = 128 * 128;    // 64 columns of a tile: 128 rows of 128 bytes
// TMEM columns: S (and P over its first half) and O of the two tiles
constexpr uint32_t kS = 0, kO = 256;

template <int D>
struct Layout {
    static constexpr uint32_t tile = D / 64 * kHalf;
    static constexpr uint32_t q = 0;                     // two tiles
    static constexpr uint32_t k = 2 * tile, v = 4 * tile;   // two stages each
    static constexpr uint32_t scales = 6 * tile;
    static constexpr uint32_t bytes = scales + 1024 + 1024;  // scales, barriers; alignment
};

// Of a step's eight groups of 16 tokens: factor and offset of their scores, and what their
// weights count in the sum.
struct Scales {
    float k[8], log_v[8], inv_v[8];
};

struct Shared {
    Scales scales[4];                    // of step i at i & 3
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t fin;
    uint32_t tmem;
    volatile int abort;
};
static_assert(sizeof(Shared) <= 1024, "scales and barriers");

struct Job {
    int request, head;
    int tokens, row0, rows;              // cached; first row of the request's, and how many
    int hidden;                          // keys that the request's row 0 sees
    int64_t token0;                      // of the packed q
};

// The rows' tiles of the requests that this kernel takes, last ones first: later tokens see more
// keys, and the long tiles start early.
__device__ __forceinline__ bool job_of(const CacheAttention& p, int index, int head, Job& job) {
    __shared__ int64_t sums[kThreads / 32];
    __shared__ Job found;
    __shared__ int any;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int k = (p.N + kThreads - 1) / kThreads;
    const int i0 = threadIdx.x * k, i1 = i0 + k < p.N ? i0 + k : p.N;
    auto rows_of = [&](int i, int64_t& bos) {
        int64_t eos;
        if (p.cu) {
            clamped_seq(p.cu, i, p.N, p.T, bos, eos);
        } else {
            bos = i;
            eos = i + 1;
        }
        const int64_t rows = (eos - bos) * p.group;
        return rows >= p.many_rows ? rows : 0;
    };
    int64_t mine = 0, bos;
    for (int i = i0; i < i1; ++i) mine += (rows_of(i, bos) + 2 * kRows - 1) / (2 * kRows);
    int64_t x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sums[w] = x;
    if (threadIdx.x == 0) any = 0;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        before += i < w ? sums[i] : 0;
        total += sums[i];
    }
    int64_t at = before + x - mine;
    const int64_t want = total - 1 - index;
    if (want >= at && want < at + mine) {
        for (int i = i0; i < i1; ++i) {
            const int64_t rows = rows_of(i, bos), tiles = (rows + 2 * kRows - 1) / (2 * kRows);
            if (want < at + tiles) {
                const int64_t table = (int64_t)p.width << p.block_log2;
                const int64_t most = table < 0x7fff0000 ? table : 0x7fff0000;
                const int64_t c = p.context[i], r0 = (want - at) * 2 * kRows;
                found.request = i;
                found.head = head;
                found.tokens = (int)(c < 0 ? 0 : (c < most ? c : most));
                found.row0 = (int)r0;
                found.rows = (int)(rows - r0 < 2 * kRows ? rows - r0 : 2 * kRows);
                found.hidden = found.tokens - (int)(rows / p.group) + 1;
                found.token0 = bos;
                any = 1;
                break;
            }
            at += tiles;
        }
    }
    __syncthreads();
    job = found;
    return any != 0;
}

// ------------------------------------------------------------------- waits
// Bounded: asleep in the barrier up to 20 us at a time, 2^19 times at most.
__device__ __forceinline__ bool sleep_wait(Shared* s, uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_u32(bar);
    for (uint32_t i = 0; i < (1u << 19); ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(at), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
        if (s->abort) return false;
    }
    return false;
}

// A whole warp's: all lanes go on, or none, and then every role leaves its loop.
__device__ __forceinline__ bool wait_warp(const CacheAttention& p, Shared* s, uint64_t* bar,
                                          uint32_t parity, int site) {
    const bool ok = sleep_wait(s, bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    atomicCAS(p.status, 0, site);
    s->abort = 1;
    return false;
}

__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---------------------------------------------------------------- products
// Low words of the operands' descriptors; the high word (128-byte swizzle, 1024 bytes between
// groups of 8 rows) is the same for all.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
// K-major: rows of 64 channels; step kk covers 16 channels.
__device__ __forceinline__ uint32_t tile_k(uint32_t tile) { return tile >> 4 | 1u << 16; }
__device__ __forceinline__ constexpr uint32_t step_k(int kk) {
    return ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
}
// MN-major: rows are the summed index; step kk covers 16 rows.
__device__ __forceinline__ uint32_t tile_mn(uint32_t tile) { return tile >> 4 | (kHalf >> 4) << 16; }
__device__ __forceinline__ constexpr uint32_t step_mn(int kk) { return kk * 2048 >> 4; }

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
    return idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

// D (+)= A B, one step of 16: A in shared memory, or in TMEM.  The whole warp calls it and one
// lane (always the same) issues.
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b, uint32_t id, int add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %4};\n\t"
        "mov.b64 b, {%2, %4};\n\tsetp.ne.b32 p, %5, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(kDescHigh), "r"(add)
        : "memory");
}
__device__ __forceinline__ void product_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t id,
                                           int add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %4};\n\t"
        "setp.ne.b32 p, %5, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(kDescHigh), "r"(add)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::
            "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float exp2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ------------------------------------------------------------------ issuing
template <int D>
__device__ __forceinline__ void issue(const CacheAttention& p, Shared* s, uint32_t base, int steps,
                                      int tiles) {
    using L = Layout<D>;
    constexpr uint32_t id_s = idesc_f16(128, kTokens, 0, 0), id_o = idesc_f16(128, D, 0, 1);
    auto scores = [&](int t, int i) {
        const uint32_t q = tile_k(base + L::q + t * L::tile);
        const uint32_t k = tile_k(base + L::k + (i & 1) * L::tile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            product(kS + 128 * t, q + step_k(kk), k + step_k(kk), id_s, kk > 0);
        }
        commit(&s->s_full[t]);
    };
    bool ok = wait_warp(p, s, &s->k_full[0], 0, 401);
    if (ok) {
        fence_proxy_async();
        tc_fence_after();
        for (int t = 0; t < tiles; ++t) scores(t, 0);
        commit(&s->k_empty[0]);
    }
    for (int i = 0; ok && i < steps; ++i) {
        const int stage = i & 1, phase = (i >> 1) & 1;
        for (int t = 0; ok && t < tiles; ++t) {
            ok = (t > 0 || wait_warp(p, s, &s->v_full[stage], phase, 402)) &&
                 wait_warp(p, s, &s->p_full[t], i & 1, 403);
            if (!ok) break;
            fence_proxy_async();
            tc_fence_after();
            const uint32_t v = tile_mn(base + L::v + stage * L::tile);
#pragma unroll
            for (int kk = 0; kk < kTokens / 16; ++kk) {
                product_ta(kO + 128 * t, kS + 128 * t + 8 * kk, v + step_mn(kk), id_o,
                           i > 0 || kk > 0);
            }
            commit(&s->o_full[t]);
            if (i + 1 < steps) {
                // the next scores overwrite P: its products have to be done
                ok = wait_warp(p, s, &s->o_full[t], i & 1, 404) &&
                     (t > 0 || wait_warp(p, s, &s->k_full[stage ^ 1], ((i + 1) >> 1) & 1, 405));
                if (!ok) break;
                fence_proxy_async();
                tc_fence_after();
                scores(t, i + 1);
            }
        }
        if (!ok) break;
        commit(&s->v_empty[stage]);
        if (i + 1 < steps) commit(&s->k_empty[stage ^ 1]);
    }
    commit(&s->fin);
    mbar_wait(&s->fin, 0, nullptr);      // no product outlives the CTA
}

// ------------------------------------------------------------------ filling
// 16 channels of one token from e4m3 to two vectors of fp16 in a tile.
__device__ __forceinline__ void spread(uint8_t* tile, int row, int part, const uint4& raw) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint4 h[2];
    h[0] = make_uint4(half2_of_e4m3(w[0]), half2_of_e4m3_high(w[0]), half2_of_e4m3(w[1]),
                      half2_of_e4m3_high(w[1]));
    h[1] = make_uint4(half2_of_e4m3(w[2]), half2_of_e4m3_high(w[2]), half2_of_e4m3(w[3]),
                      half2_of_e4m3_high(w[3]));
    // parts 0-3 and 4-7 of a row lie in two halves of the same banks: they take their two
    // vectors in opposite order
    const int first = part >> 2;
    uint8_t* half = tile + first * kHalf + row * 128;
    const int chunk = 2 * (part & 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = i ^ first;
        *reinterpret_cast<uint4*>(half + (((chunk + j) ^ (row & 7)) << 4)) = j ? h[1] : h[0];
    }
}

template <int D>
__device__ __forceinline__ void fill(const CacheAttention& p, const Job& job, Shared* s,
                                     uint8_t* sm, int steps, int high) {
    using L = Layout<D>;
    constexpr int kParts = D / 16;                       // vectors of 16 numbers in a row
    constexpr int kPass = 32 * kFillWarps / kParts;      // rows of all threads' loads
    constexpr int kLoads = kTokens / kPass;
    const int tid = threadIdx.x - 32 * kSoftWarps, lane = tid & 31;
    const int part = tid % kParts, row0 = tid / kParts;
    const int32_t* table = p.table + (int64_t)job.request * p.width;
    // lanes 0-7: the blocks of a step's groups of 16 tokens (-1: not there), and their scales
    auto blocks_of = [&](int i) {
        const int token = i * kTokens + 16 * (lane & 7);
        int b = -1;
        if (i < steps && token < high) {
            b = table[token >> p.block_log2];
            if (b >= p.num_blocks) b = -1;
        }
        return b < 0 ? -1 : b;
    };
    auto load = [&](const uint8_t* cache, int i, int blocks, uint4 (&raw)[kLoads]) {
#pragma unroll
        for (int r = 0; r < kLoads; ++r) {
            const int row = row0 + r * kPass, token = i * kTokens + row;
            const int b = __shfl_sync(0xffffffffu, blocks, row >> 4);
            raw[r] = make_uint4(0, 0, 0, 0);
            if (b >= 0 && token < high) {
                const int64_t at = (((int64_t)b * p.heads + job.head) << p.block_log2) +
                                   (token & ((1 << p.block_log2) - 1));
                raw[r] = *reinterpret_cast<const uint4*>(cache + at * D + 16 * part);
            }
        }
    };
    auto store = [&](uint8_t* tile, const uint4 (&raw)[kLoads]) {
#pragma unroll
        for (int r = 0; r < kLoads; ++r) spread(tile, row0 + r * kPass, part, raw[r]);
    };
    uint4 k[kLoads], v[kLoads];
    int blocks = blocks_of(0), next = blocks_of(1);
    load(p.k_cache, 0, blocks, k);
    for (int i = 0; i < steps; ++i) {
        const int stage = i & 1, phase = ((i >> 1) & 1) ^ 1;
        load(p.v_cache, i, blocks, v);
        float ks = 0.0f, log_v = kNone, inv_v = 0.0f;
        if (tid < 8 && blocks >= 0) {
            const int64_t at = (int64_t)blocks * p.heads + job.head;
            const float vs = p.v_scale[at];
            ks = p.k_scale[at];
            log_v = __log2f(vs);
            inv_v = __frcp_rn(vs);
        }
        if (i > 1 && !wait_warp(p, s, &s->k_empty[stage], phase, 411)) return;
        store(sm + L::k + stage * L::tile, k);
        if (tid < 8) {
            Scales& to = s->scales[i & 3];
            to.k[tid] = ks;
            to.log_v[tid] = log_v;
            to.inv_v[tid] = inv_v;
        }
        arrive_warp(&s->k_full[stage]);
        if (i + 1 < steps) load(p.k_cache, i + 1, next, k);
        if (i > 1 && !wait_warp(p, s, &s->v_empty[stage], phase, 412)) return;
        store(sm + L::v + stage * L::tile, v);
        arrive_warp(&s->v_full[stage]);
        blocks = next;
        next = blocks_of(i + 2);
    }
}

// ------------------------------------------------------------------ softmax
template <bool MASKED>
__device__ __forceinline__ float largest(const uint32_t (&r)[16], int seen) {
    float top = kNone;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float x = __uint_as_float(r[j]);
        top = fmaxf(top, MASKED && j >= seen ? kNone : x);
    }
    return top;
}

// 16 scores to weights, as pairs; their sum.
template <bool MASKED>
__device__ __forceinline__ float weights(const uint32_t (&r)[16], float f, float offset, int seen,
                                         uint32_t* pairs) {
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        float e[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            e[n] = exp2_of(fmaf(__uint_as_float(r[j + n]), f, offset));
            if (MASKED && j + n >= seen) e[n] = 0.0f;
            sum[n] += e[n];
        }
        pairs[j / 2] = half2_of(e[0], e[1]);
    }
    return sum[0] + sum[1];
}

template <int D>
__device__ __forceinline__ void soften(const CacheAttention& p, const Job& job, Shared* s,
                                       uint8_t* sm, int steps, int t, float factor) {
    const int row = threadIdx.x & 127, lanes_of = (threadIdx.x >> 5) & 3;
    const uint32_t lane0 = (uint32_t)lanes_of << 21;     // TMEM lane 32 * (warp % 4)
    const uint32_t cs = lane0 + kS + 128 * t, co = lane0 + kO + 128 * t;
    const int flat = job.row0 + kRows * t + row, limit = job.hidden + flat / p.group;
    // the first row of this warp sees the fewest keys
    const int fewest = job.hidden + (flat - (threadIdx.x & 31)) / p.group;
    float m = kNone, l = 0.0f;
    bool ok = true;
    for (int i = 0; i < steps; ++i) {
        const int first = i * kTokens, seen = limit - first;
        const bool masked = first + kTokens > fewest;
        // (the scales were written before the keys that the scores are of)
        ok = wait_warp(p, s, &s->s_full[t], i & 1, 422);
        if (!ok) break;
        tc_fence_after();
        const Scales& sc = s->scales[i & 3];
        float top = kNone;
#pragma unroll
        for (int g = 0; g < 8; g += 2) {
            uint32_t r[2][16];
            tmem_ld16(cs + 16 * g, r[0]);
            tmem_ld16(cs + 16 * g + 16, r[1]);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float x = masked ? largest<true>(r[h], seen - 16 * (g + h))
                                       : largest<false>(r[h], 16);
                // (the factor of a block that is not there is 0: no score of it counts)
                const float y = fmaf(x, factor * sc.k[g + h], sc.log_v[g + h]);
                top = fmaxf(top, x == kNone ? kNone : y);
            }
        }
        const bool raise = top > m + kSlack;
        if (__any_sync(0xffffffffu, raise)) {
            const float now = fmaxf(m, top), less = now > m ? exp2_of(m - now) : 1.0f;
            m = now;
            l *= less;
            if (i > 0) {
                ok = wait_warp(p, s, &s->o_full[t], (i - 1) & 1, 423);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t r[2][16];
                    tmem_ld16(co + c, r[0]);
                    tmem_ld16(co + c + 16, r[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        r[0][j] = __float_as_uint(__uint_as_float(r[0][j]) * less);
                        r[1][j] = __float_as_uint(__uint_as_float(r[1][j]) * less);
                    }
                    tmem_st16(co + c, r[0]);
                    tmem_st16(co + c + 16, r[1]);
                }
            }
        }
        const float ref = (m == kNone ? 0.0f : m) - kRaise;
#pragma unroll
        for (int g = 0; g < 8; g += 2) {
            uint32_t r[2][16], pairs[16];
            tmem_ld16(cs + 16 * g, r[0]);
            tmem_ld16(cs + 16 * g + 16, r[1]);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float f = factor * sc.k[g + h], offset = sc.log_v[g + h] - ref;
                const float sum = masked
                    ? weights<true>(r[h], f, offset, seen - 16 * (g + h), pairs + 8 * h)
                    : weights<false>(r[h], f, offset, 16, pairs + 8 * h);
                l = fmaf(sum, sc.inv_v[g + h], l);
            }
            tmem_st16(cs + 8 * g, pairs);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&s->p_full[t]);
    }
    if (ok && steps > 0) ok = wait_warp(p, s, &s->o_full[t], (steps - 1) & 1, 424);
    tc_fence_after();
    const bool mine = ok && kRows * t + row < job.rows;
    const float by = l == 0.0f ? 0.0f : 1.0f / l;
    const int j = flat / p.group;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) +
                         ((job.token0 + j) * (p.heads * p.group) + job.head * p.group + flat -
                          j * p.group) * D;
#pragma unroll
    for (int c = 0; c < D; c += 32) {
        uint32_t r[2][16];
        if (steps > 0) {
            tmem_ld16(co + c, r[0]);
            tmem_ld16(co + c + 16, r[1]);
            tmem_wait_ld();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float lo = l == 0.0f ? 0.0f : __uint_as_float(r[h][2 * i]) * by;
                const float hi = l == 0.0f ? 0.0f : __uint_as_float(r[h][2 * i + 1]) * by;
                const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            if (mine) {
                uint4* to = reinterpret_cast<uint4*>(out + c + 16 * h);
                to[0] = make_uint4(w[0], w[1], w[2], w[3]);
                to[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    }
}

// This thread's row of q, scaled to [1, 2) and in fp16, into its tile; the factor of its scores.
template <int D>
__device__ __forceinline__ float stage_query(const CacheAttention& p, const Job& job, uint8_t* sm) {
    const int row = threadIdx.x & 127, t = threadIdx.x >> 7, n = kRows * t + row;
    const int flat = job.row0 + n, j = flat / p.group;
    const bool there = n < job.rows;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                             (job.token0 + j) * p.q_stride +
                             (int64_t)(job.head * p.group + flat - j * p.group) * D;
    uint4 raw[D / 8];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        raw[i] = there ? *reinterpret_cast<const uint4*>(q + 8 * i) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[e] << 16)),
                                   fabsf(__uint_as_float(w[e] & 0xffff0000u))));
        }
    }
    int e = __float_as_int(top) >> 23;
    e = e < 1 ? 1 : (e > 253 ? 253 : e);
    // a negative scale turns q around, so that the largest score is the largest product
    const float down = copysignf(__int_as_float((254 - e) << 23), p.scale);
    uint8_t* tile = sm + Layout<D>::q + t * Layout<D>::tile;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = half2_of(__uint_as_float(w[k] << 16) * down,
                            __uint_as_float(w[k] & 0xffff0000u) * down);
        }
        *reinterpret_cast<uint4*>(tile + (i >> 3) * kHalf + row * 128 +
                                  (((i & 7) ^ (row & 7)) << 4)) =
            make_uint4(h[0], h[1], h[2], h[3]);
    }
    return __int_as_float(e << 23) * (fabsf(p.scale) * 1.44269504088896340736f);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cache_prompt_kernel(CacheAttention p) {
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                             ~(uintptr_t)1023);
    Shared* s = reinterpret_cast<Shared*>(sm + Layout<D>::scales);
    const int w = threadIdx.x >> 5;
    // (the earliest any CTA can report a wait is seconds away)
    if (p.clears && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    Job job;
    if (!job_of(p, blockIdx.x / p.heads, blockIdx.x % p.heads, job)) return;
    if (threadIdx.x == 32 * kIssueWarp) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->k_full[i], kFillWarps);
            mbar_init(&s->v_full[i], kFillWarps);
            mbar_init(&s->k_empty[i], 1);
            mbar_init(&s->v_empty[i], 1);
            mbar_init(&s->s_full[i], 1);
            mbar_init(&s->p_full[i], kSoftWarps / 2);
            mbar_init(&s->o_full[i], 1);
        }
        mbar_init(&s->fin, 1);
        s->abort = 0;
        fence_mbar_init();
    }
    if (w == kIssueWarp) {
        __syncwarp();
        tmem_alloc(&s->tmem, 512);
        tmem_relinquish();
    }
    float factor = 0.0f;
    if (w < kSoftWarps) factor = stage_query<D>(p, job, sm);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int tiles = job.rows > kRows ? 2 : 1;
    const int high = job.hidden + (job.row0 + job.rows - 1) / p.group;
    const int steps = high > 0 ? (high + kTokens - 1) / kTokens : 0;
    if (w < kSoftWarps) {
        const int t = threadIdx.x >> 7;
        if (t < tiles) soften<D>(p, job, s, sm, steps, t, factor);
    } else if (w < kIssueWarp) {
        fill<D>(p, job, s, sm, steps, high);
    } else if (steps > 0) {
        issue<D>(p, s, smem_u32(sm), steps, tiles);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == kIssueWarp) tmem_dealloc(s->tmem, 512);
}

template <int D>
cudaError_t launch_dim(const CacheAttention& p, cudaStream_t stream) {
    const cudaError_t err = cudaFuncSetAttribute(
        cache_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::bytes);
    if (err != cudaSuccess) return err;
    // every request may leave a tile partly filled
    const int64_t rows = (int64_t)p.T * p.group;
    const int64_t tiles = rows / (2 * kRows) + (p.N < p.T ? p.N : p.T);
    if (tiles * p.heads > 0x7fffffff) return cudaErrorInvalidValue;
    cache_prompt_kernel<D><<<(unsigned)(tiles * p.heads), kThreads, Layout<D>::bytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool cache_prompt_takes(int32_t d, int dtype) { return dtype == 1 && (d == 64 || d == 128); }

cudaError_t launch_cache_prompt(const CacheAttention& p, cudaStream_t stream) {
    return p.d == 64 ? launch_dim<64>(p, stream) : launch_dim<128>(p, stream);
}

}  // namespace kda
