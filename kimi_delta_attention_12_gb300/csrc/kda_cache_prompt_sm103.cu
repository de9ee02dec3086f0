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
// A CTA stays on its SM and takes its share of all steps, a stretch that may begin and end inside
// an item; such an item's sums are joined by a second kernel.
//
// The tiles take turns: while one's softmax runs, the tensor core works for the other.  Roles:
// warps 0-7 a row each (softmax, the output), warps 8-11 read e4m3 tiles of the cache and write
// them as fp16 (exact) in the operands' layout, warps 12 and 13 issue the products of a tile
// each, warps 14 and 15 only give their registers away.
//
// fp16, not bf16: e4m3 numbers are fp16 numbers, and so are the channels of a bf16 query, down to
// 2^-31 of its largest, which a power of two per row brings to [2^14, 2^15); and P keeps 11 bits.
// Scales of key blocks go into the exponent's factor, those of value blocks into its offset, as in
// the kernel for few rows: p' = 2^(s - m + 7) v_scale with m at most 8 below the running maximum of
// s + log2 v_scale.  That slack is what spares most tiles the rescaling of O: it is done where the
// maximum has grown by more, and P stays below 2^15 (a slack of 4 took 850 us where this one takes
// 836).  What is 2^-21 of the heaviest or more keeps all its bits.
//
// Measured: 4,096 new tokens behind 12,288, 32 heads over 8, d = 128: 836 us, 1.15 PFLOP/s, 60 % of
// the measured bf16 rate.  The tensor pipe is busy for 46 % of the cycles and so are the issue
// slots; what bounds it is the chain scores - softmax - products of each tile, some 3,600 cycles a
// step against 2,048 of products for both tiles: without exponentials, maxima, cache loads and
// seven of eight products, in a copy made for timing, the hand-overs alone took 590 us.  Two warps to
// 32 rows instead of one (16 softmax warps) took 1,035, scores read twice instead of held in
// registers the same as now, the two tiles side by side instead of half a step apart 4 % more.  The
// chain is that of this order of roles: P lies over S, so a tile's next scores wait for the products of
// its weights.  The same at d = 64: 721 us, 35 % of the rate, for half of the operations.  The
// compiler spills some 200 bytes a thread (204 stored, 356 loaded).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kda_cache.h"
#include "kda_e4m3.cuh"
#include "kda_follow.cuh"
#include "kda_packed.cuh"
#include "kda_seqlens.cuh"
#include "sm103_ptx.cuh"

namespace kda {
namespace {

using namespace sm103;

constexpr int kRows = 128;               // of a tile
constexpr int kTokens = 128;             // of a step
constexpr int kSoftWarps = 8, kFillWarps = 4;
constexpr int kIssueWarp = kSoftWarps + kFillWarps;
constexpr int kThreads = 32 * (kIssueWarp + 4);   // whole groups of four warps share registers
// Registers of a thread: at launch, and then of the softmax, filling and issuing groups.
constexpr int kRegs = 128, kSoftRegs = 176, kFillRegs = 120, kIssueRegs = 40;
static_assert(2 * kSoftRegs + kFillRegs + kIssueRegs <= 4 * kRegs, "register split");
static_assert(kSoftRegs >= kRegs && kFillRegs <= kRegs && kIssueRegs <= kRegs,
              "a group that gives registers away ends with no more than it had");
constexpr float kNone = -INFINITY;
constexpr float kSlack = 8.0f, kRaise = 7.0f;
constexpr int kLeastSteps = 8;           // of a block, so that parts are worth their joining
// What an item's start and end take, and the joining of parts, in steps.
constexpr int kStart = 3;
__host__ __device__ constexpr int join_steps(int d) { return d == 128 ? 12 : 8; }
constexpr int kJoinThreads = 256, kJoinRows = 32;
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

// Of a group of 16 tokens: factor and offset of their scores, and what their weights count in
// the sum.
struct __align__(16) Scales {
    float k, log_v, inv_v, unused;
};

struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], p_full[2][2], o_full[2];   // p_full: of each half of the weights
    uint64_t fin[2];
    uint64_t go;                         // the second tile sets out when the first has its weights
};

struct Shared {
    Scales scales[4][8];                 // of step i at i & 3
    Bars bars[2];                        // of one piece of work and the next
    uint32_t tmem;
    volatile int abort;
};
static_assert(sizeof(Shared) <= 1024, "scales and barriers");

// 256 rows of a request and head, and the steps that they need.
struct Item {
    int request, head;
    int tokens, row0, rows;              // cached; first row of the request's, and how many
    int hidden;                          // keys that the request's row 0 sees
    int64_t token0;                      // of the packed q
    int64_t begin;                       // where its steps begin among all
    int nominal, steps;                  // steps set aside, those that its last row needs
};

// Every tile of a request counts as many steps as its last one needs, so that a step's place is
// found without walking the tiles; a tile that sees fewer keys leaves the rest of its steps empty.
struct Span {
    int64_t bos, rows, tiles, all;
    int tokens, nominal;
};

__device__ __forceinline__ Span span_of(const CacheAttention& p, int i) {
    Span s;
    int64_t eos;
    if (p.cu) {
        clamped_seq(p.cu, i, p.N, p.T, s.bos, eos);
    } else {
        s.bos = i;
        eos = i + 1;
    }
    const int64_t table = (int64_t)p.width << p.block_log2;
    const int64_t most = table < 0x7fff0000 ? table : 0x7fff0000;
    const int64_t c = p.context[i];
    s.tokens = (int)(c < 0 ? 0 : (c < most ? c : most));
    s.rows = (eos - s.bos) * p.group;
    if (s.rows < p.many_rows) s.rows = 0;
    s.tiles = (s.rows + 2 * kRows - 1) / (2 * kRows);
    s.nominal = s.tokens > 0 ? (int)(((int64_t)s.tokens + kTokens - 1) / kTokens) : 1;
    s.all = s.tiles * p.heads * s.nominal;
    return s;
}

// What each block takes: the steps begin .. end - 1 of all, from request `request` on, whose
// steps begin at `first`.  All threads of the block call it.
struct Stretch {
    int64_t begin, end, per, first;
    int request;
};

template <int THREADS>
__device__ __forceinline__ Stretch stretch_of(const CacheAttention& p, int block, int blocks) {
    __shared__ int64_t sums[THREADS / 32], items_of[THREADS / 32];
    __shared__ int longest_of[THREADS / 32];
    __shared__ int64_t found_first;
    __shared__ int found;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int k = (p.N + THREADS - 1) / THREADS;
    const int i0 = threadIdx.x * k, i1 = i0 + k < p.N ? i0 + k : p.N;
    int64_t mine = 0, items = 0;
    int longest = 0;
    for (int i = i0; i < i1; ++i) {
        const Span s = span_of(p, i);
        mine += s.all;
        items += s.tiles * p.heads;
        if (s.tiles > 0 && s.nominal > longest) longest = s.nominal;
    }
    int64_t x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
        items += __shfl_xor_sync(0xffffffffu, items, d);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) {
        sums[w] = x;
        items_of[w] = items;
        longest_of[w] = longest;
    }
    if (threadIdx.x == 0) found = -1;
    __syncthreads();
    int64_t total = 0, before = 0;
    items = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        before += i < w ? sums[i] : 0;
        total += sums[i];
        items += items_of[i];
        longest = max(longest, longest_of[i]);
    }
    // Even stretches, or stretches of whole items (whole where all are equally long): by what the
    // last block to end has to do.  32 heads over 8, d = 128, us, even against whole: 512, 2,000
    // new tokens 39 against 32, 83 against 68; 1,000 behind 3,000 101 against 86; finding this out
    // takes 2 where stretches stay even.
    Stretch s;
    s.per = (total + blocks - 1) / blocks;
    const int64_t rounds = (items + blocks - 1) / blocks, whole = rounds * longest;
    const int64_t cut = s.per + (total > 0 ? (s.per / longest + 1) * kStart : 0) + join_steps(p.d);
    if (s.per < kLeastSteps) s.per = kLeastSteps;
    if (whole > 0 && whole + rounds * kStart <= cut) s.per = whole;
    s.begin = s.per * block;
    s.end = s.begin + s.per < total ? s.begin + s.per : total;
    int64_t at = before + x - mine;
    if (s.begin < total && at <= s.begin && s.begin < at + mine) {
        for (int i = i0; i < i1; ++i) {
            const int64_t all = span_of(p, i).all;
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

// The item of step `at`, from request i on, whose steps begin at `first`.  Tiles follow each other
// first, last, second, last but one, ...: under a causal mask a tile and its neighbour together
// take the same time wherever they stand.
__device__ __forceinline__ Item item_at(const CacheAttention& p, int64_t at, int& i,
                                        int64_t& first) {
    Span s = span_of(p, i);
    while (at >= first + s.all && i + 1 < p.N) {
        first += s.all;
        s = span_of(p, ++i);
    }
    const int64_t n = (at - first) / s.nominal, head = n / s.tiles, k = n - head * s.tiles;
    const int64_t row0 = 2 * kRows * (k & 1 ? s.tiles - 1 - (k >> 1) : k >> 1);
    Item t;
    t.request = i;
    t.head = (int)head;
    t.tokens = s.tokens;
    t.row0 = (int)row0;
    t.rows = (int)(s.rows - row0 < 2 * kRows ? s.rows - row0 : 2 * kRows);
    t.hidden = s.tokens - (int)(s.rows / p.group) + 1;
    t.token0 = s.bos;
    t.begin = first + n * s.nominal;
    t.nominal = s.nominal;
    const int high = t.hidden + (t.row0 + t.rows - 1) / p.group;
    t.steps = high > kTokens ? (high + kTokens - 1) / kTokens : 1;
    return t;
}

// Where block `block` leaves its sums of an item that it does not have whole: the one that it
// begins with, or another.
__device__ __forceinline__ float* part_of(const CacheAttention& p, int64_t block, bool begins_with,
                                          int D) {
    return p.prompt_partial + (block * 2 + !begins_with) * (2 * kRows) * (D + 2);
}

template <int N>
__device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------- waits
// Bounded (mbar_wait), a whole warp's: all lanes go on, or none, and then every role leaves its
// loop.  Polls that sleep in the barrier for as long as they are let (a time of 20 us) were
// slower to wake: 837 -> 858 us.
__device__ __forceinline__ bool wait_warp(const CacheAttention& p, Shared* s, uint64_t* bar,
                                          uint32_t parity, int site) {
    const bool ok = mbar_wait(bar, parity, &s->abort);
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
// All products of tile t.
template <int D>
__device__ __forceinline__ void issue(const CacheAttention& p, Shared* s, Bars* b, uint32_t base,
                                      int steps, int t) {
    using L = Layout<D>;
    constexpr uint32_t id_s = idesc_f16(128, kTokens, 0, 0), id_o = idesc_f16(128, D, 0, 1);
    const uint32_t q = tile_k(base + L::q + t * L::tile), cs = kS + 128 * t, co = kO + 128 * t;
    for (int i = -1; i < steps; ++i) {
        if (i >= 0) {
            const uint32_t v = tile_mn(base + L::v + (i & 1) * L::tile);
            if (!wait_warp(p, s, &b->v_full[i & 1], (i >> 1) & 1, 402)) break;
            fence_proxy_async();
            bool ok = true;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!(ok = ok && wait_warp(p, s, &b->p_full[t][h], i & 1, 403))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 4 * h; kk < 4 * h + 4; ++kk) {
                    product_ta(co, cs + 8 * kk, v + step_mn(kk), id_o, i > 0 || kk > 0);
                }
            }
            if (!ok) break;
            commit(&b->o_full[t]);
            commit(&b->v_empty[i & 1]);
        }
        if (i + 1 < steps) {
            // Half a step behind: one tile's softmax then runs beside the other's products.  Side
            // by side they contend for the issue slots and then for the tensor core.
            if (i < 0 && t == 1 && !wait_warp(p, s, &b->go, 0, 406)) break;
            const int stage = (i + 1) & 1;
            const uint32_t k = tile_k(base + L::k + stage * L::tile);
            if (!wait_warp(p, s, &b->k_full[stage], ((i + 1) >> 1) & 1, 401)) break;
            fence_proxy_async();
            // the scores overwrite P: its products have to be done
            if (i >= 0 && !wait_warp(p, s, &b->o_full[t], i & 1, 404)) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                product(cs, q + step_k(kk), k + step_k(kk), id_s, kk > 0);
            }
            commit(&b->s_full[t]);
            commit(&b->k_empty[stage]);
        }
    }
    commit(&b->fin[t]);
    mbar_wait(&b->fin[t], 0, nullptr);   // no product outlives the CTA
}

// ------------------------------------------------------------------ filling
// A load that stays where it is written, ahead of the waits that it is to pass by.
__device__ __forceinline__ uint4 load_early(const uint8_t* p) {
    uint4 r;
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// 16 channels of one token from e4m3 to two neighbouring vectors of fp16.
__device__ __forceinline__ void spread(uint8_t* tile, uint32_t at, const uint4& raw) {
    *reinterpret_cast<uint4*>(tile + at) =
        make_uint4(half2_of_e4m3(raw.x), half2_of_e4m3_high(raw.x), half2_of_e4m3(raw.y),
                   half2_of_e4m3_high(raw.y));
    *reinterpret_cast<uint4*>(tile + (at ^ 16)) =
        make_uint4(half2_of_e4m3(raw.z), half2_of_e4m3_high(raw.z), half2_of_e4m3(raw.w),
                   half2_of_e4m3_high(raw.w));
}

// Steps first .. first + steps - 1 of an item.
template <int D>
__device__ __forceinline__ void fill(const CacheAttention& p, const Item& job, Shared* s, Bars* bars,
                                     uint8_t* sm, int first, int steps, int high) {
    using L = Layout<D>;
    constexpr int kParts = D / 16;                       // vectors of 16 numbers in a row
    constexpr int kPass = 32 * kFillWarps / kParts;      // rows of all threads' loads
    constexpr int kLoads = kTokens / kPass;
    const int tid = threadIdx.x - 32 * kSoftWarps, lane = tid & 31;
    // Eight lanes, which store at once, have four parts of two rows each: their 16-byte vectors lie
    // in eight different places of a row's 128 bytes.
    const int part = D == 64 ? lane & 3 : (lane & 3) + ((lane >> 1) & 4);
    const int row0 = D == 64 ? tid >> 2 : 4 * (tid >> 5) + 2 * (lane >> 4) + ((lane >> 2) & 1);
    const uint32_t at0 = (part >> 2) * kHalf + row0 * 128 + (((2 * (part & 3)) ^ (row0 & 7)) << 4);
    const int32_t* table = p.table + (int64_t)job.request * p.width;
    const int mask = (1 << p.block_log2) - 1;
    const uint32_t block_bytes = (uint32_t)p.heads * D << p.block_log2;
    const uint32_t in_block = ((uint32_t)job.head * D << p.block_log2) + 16 * part;
    // lanes 0-7: the blocks of a step's groups of 16 tokens, -1 where there is none
    auto blocks_of = [&](int i) {
        const int token = (first + i) * kTokens + 16 * (lane & 7);
        const int b = i < steps && token < high ? table[token >> p.block_log2] : -1;
        return b >= 0 && b < p.num_blocks ? b : -1;
    };
    // Rows that are not there are read from block 0, so that no load waits for a branch, and
    // zeroed.
    auto load = [&](const uint8_t* cache, int i, int blocks, uint4 (&raw)[kLoads]) {
#pragma unroll
        for (int r = 0; r < kLoads; ++r) {
            const int row = row0 + r * kPass, token = (first + i) * kTokens + row;
            const int b = max(__shfl_sync(0xffffffffu, blocks, row >> 4), 0);
            raw[r] = load_early(cache + (uint64_t)(uint32_t)b * block_bytes +
                                (in_block + (token & mask) * D));
        }
    };
    auto store = [&](uint8_t* tile, int i, int blocks, uint4 (&raw)[kLoads]) {
        // (whole steps, but for a request's last)
        if (__any_sync(0xffffffffu, blocks < 0) || (first + i + 1) * kTokens > high) {
#pragma unroll
            for (int r = 0; r < kLoads; ++r) {
                const int row = row0 + r * kPass;
                const int b = __shfl_sync(0xffffffffu, blocks, row >> 4);
                if (b < 0 || (first + i) * kTokens + row >= high) raw[r] = make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int r = 0; r < kLoads; ++r) spread(tile, at0 + r * kPass * 128, raw[r]);
    };
    // of this lane's group: the scales of keys and values
    auto scales_of = [&](int blocks, float& ks, float& vs) {
        const int64_t at = (int64_t)max(blocks, 0) * p.heads + job.head;
        ks = p.k_scale[at];
        vs = p.v_scale[at];
    };
    uint4 k[kLoads], v[kLoads];
    int blocks = blocks_of(0), next = blocks_of(1);
    float ks, vs;
    load(p.k_cache, 0, blocks, k);
    scales_of(blocks, ks, vs);
    for (int i = 0; i < steps; ++i) {
        const int stage = i & 1, phase = ((i >> 1) & 1) ^ 1;
        load(p.v_cache, i, blocks, v);
        const int after = blocks_of(i + 2);
        if (i > 1 && !wait_warp(p, s, &bars->k_empty[stage], phase, 411)) return;
        store(sm + L::k + stage * L::tile, i, blocks, k);
        if (tid < 8) {
            // not there: no score of it counts
            Scales& to = s->scales[i & 3][tid];
            to.k = blocks < 0 ? 1.0f : ks;
            to.log_v = blocks < 0 ? kNone : __log2f(vs);
            to.inv_v = blocks < 0 ? 0.0f : __frcp_rn(vs);
        }
        arrive_warp(&bars->k_full[stage]);
        load(p.k_cache, i + 1, next, k);
        scales_of(next, ks, vs);
        if (i > 1 && !wait_warp(p, s, &bars->v_empty[stage], phase, 412)) return;
        store(sm + L::v + stage * L::tile, i, blocks, v);
        arrive_warp(&bars->v_full[stage]);
        blocks = next;
        next = after;
    }
}

// ------------------------------------------------------------------ softmax
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}

// What a thread keeps of its row from step to step.
struct Row {
    float factor;                        // of its scores
    float m, l;                          // their reference, and the sum of weights
    int limit;                           // keys that it sees
};

// One step of a tile: weights in place of the scores.  MASKED: some rows do not see every key.
template <int D, bool MASKED>
__device__ __forceinline__ bool soften_step(const CacheAttention& p, Shared* s, Bars* b, int i,
                                            int t, uint32_t cs, uint32_t co, Row& row) {
    // (the scales were written before the keys that the scores are of)
    const Scales* sc = s->scales[i & 3];
    if (!wait_warp(p, s, &b->s_full[t], i & 1, 422)) return false;
    tc_fence_after();
    uint32_t r[kTokens];
#pragma unroll
    for (int c = 0; c < kTokens; c += 32) tmem_ld32(cs + c, r + c);
    tmem_wait_ld();
    if (MASKED) {           // scores in full, and none where the row sees nothing
        const int seen = row.limit - i * kTokens;
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            const float x = fmaf(__uint_as_float(r[j]), row.factor * sc[j / 16].k, sc[j / 16].log_v);
            r[j] = __float_as_uint(j < seen ? x : kNone);
        }
    }
    // (the groups side by side, so that no maximum waits for the one before)
    float tops[kTokens / 16];
#pragma unroll
    for (int g = 0; g < kTokens / 16; ++g) tops[g] = __uint_as_float(r[16 * g]);
#pragma unroll
    for (int j = 1; j < 15; j += 2) {
#pragma unroll
        for (int g = 0; g < kTokens / 16; ++g) {
            tops[g] = max3(tops[g], __uint_as_float(r[16 * g + j]),
                           __uint_as_float(r[16 * g + j + 1]));
        }
    }
    float top = kNone;
#pragma unroll
    for (int g = 0; g < kTokens / 16; ++g) {
        tops[g] = fmaxf(tops[g], __uint_as_float(r[16 * g + 15]));
        top = fmaxf(top, MASKED ? tops[g] : fmaf(tops[g], row.factor * sc[g].k, sc[g].log_v));
    }
    if (__any_sync(0xffffffffu, top > row.m + kSlack)) {
        const float now = fmaxf(row.m, top), less = now > row.m ? exp2_of(row.m - now) : 1.0f;
        row.m = now;
        row.l *= less;
        if (i > 0) {
            if (!wait_warp(p, s, &b->o_full[t], (i - 1) & 1, 423)) return false;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D; c += 16) {
                uint32_t x[16];
                tmem_ld16(co + c, x);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    x[j] = __float_as_uint(__uint_as_float(x[j]) * less);
                }
                tmem_st16(co + c, x);
            }
        }
    }
    const float ref = (row.m == kNone ? 0.0f : row.m) - kRaise;
#pragma unroll
    for (int h = 0; h < kTokens / 32; ++h) {
        uint64_t x[16];
        uint32_t pairs[16];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const float f = MASKED ? 1.0f : row.factor * sc[2 * h + g].k;
            const float off = (MASKED ? 0.0f : sc[2 * h + g].log_v) - ref;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = 32 * h + 16 * g + 2 * j;
                x[8 * g + j] = fma2(two(r[c], r[c + 1]), two(f, f), two(off, off));
            }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float lo, hi;
            apart(x[j], lo, hi);
            lo = exp2_of(lo);
            hi = exp2_of(hi);
            x[j] = two(lo, hi);
            pairs[j] = half2_of(lo, hi);
        }
        tmem_st16(cs + 16 * h, pairs);
        if (h & 1) {                     // half of the weights: its products may begin
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&b->p_full[t][h >> 1]);
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const uint64_t* y = x + 8 * g;
            const uint64_t sum = add2(add2(add2(y[0], y[1]), add2(y[2], y[3])),
                                      add2(add2(y[4], y[5]), add2(y[6], y[7])));
            row.l = fmaf(sum2(sum), sc[2 * h + g].inv_v, row.l);
        }
    }
    return true;
}

// Steps first .. first + steps - 1 of tile t; `part`: where to leave the sums of an item of which
// this is not all.
template <int D>
__device__ __forceinline__ void soften(const CacheAttention& p, const Item& job, Shared* s, Bars* b,
                                       int first, int steps, int t, float factor, float* part) {
    const int in_tile = threadIdx.x & 127, n = kRows * t + in_tile;
    const uint32_t lane0 = (uint32_t)(in_tile >> 5) << 21;       // TMEM lane 32 * (warp % 4)
    const uint32_t cs = lane0 + kS + 128 * t, co = lane0 + kO + 128 * t;
    const int flat = job.row0 + n, before = first * kTokens;
    Row row = {factor, kNone, 0.0f, job.hidden + flat / p.group - before};
    // the first row of this warp sees the fewest keys
    const int fewest = job.hidden + (flat - (threadIdx.x & 31)) / p.group - before;
    const int whole = fewest < 0 ? 0 : min(fewest / kTokens, steps);
    bool ok = true;
    for (int i = 0; ok && i < whole; ++i) {
        ok = soften_step<D, false>(p, s, b, i, t, cs, co, row);
        if (i == 0 && t == 0) arrive_warp(&b->go);
    }
    for (int i = whole; ok && i < steps; ++i) {
        ok = soften_step<D, true>(p, s, b, i, t, cs, co, row);
        if (i == 0 && t == 0) arrive_warp(&b->go);
    }
    ok = ok && wait_warp(p, s, &b->o_full[t], (steps - 1) & 1, 424);
    tc_fence_after();
    const bool mine = ok && n < job.rows;
    if (part) {
        if (mine) {
            part[2 * kRows * D + n] = row.m;
            part[2 * kRows * (D + 1) + n] = row.l;
        }
#pragma unroll
        for (int c = 0; c < D; c += 16) {
            uint32_t r[16];
            tmem_ld16(co + c, r);
            tmem_wait_ld();
            uint4* to = reinterpret_cast<uint4*>(part + n * D + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (mine) to[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
            }
        }
        return;
    }
    const bool none = row.l == 0.0f;         // nothing seen: O is 0 times values that may be NaN
    const float by = none ? 0.0f : 1.0f / row.l;
    const int j = flat / p.group;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) +
                         ((job.token0 + j) * (p.heads * p.group) + job.head * p.group + flat -
                          j * p.group) * D;
#pragma unroll
    for (int c = 0; c < D; c += 16) {
        uint32_t r[16], w[8];
        tmem_ld16(co + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[2 * i]) * by,
                                                           __uint_as_float(r[2 * i + 1]) * by);
            w[i] = none ? 0u : *reinterpret_cast<const uint32_t*>(&v);
        }
        if (mine) {
            uint4* to = reinterpret_cast<uint4*>(out + c);
            to[0] = make_uint4(w[0], w[1], w[2], w[3]);
            to[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

// This thread's row of q, its largest channel scaled to [2^14, 2^15), in fp16, into its tile; the
// factor of its scores.
template <int D>
__device__ __forceinline__ float stage_query(const CacheAttention& p, const Item& job, uint8_t* sm) {
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
    e = e < 15 ? 15 : (e > 254 ? 254 : e);
    // a negative scale turns q around, so that the largest score is the largest product
    const float down = copysignf(__int_as_float((268 - e) << 23), p.scale);
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
    return __int_as_float((e - 14) << 23) * (fabsf(p.scale) * 1.44269504088896340736f);
}

__device__ __forceinline__ void set_up(Bars* b, int tiles) {
    for (int i = 0; i < 2; ++i) {
        mbar_init(&b->k_full[i], kFillWarps);
        mbar_init(&b->v_full[i], kFillWarps);
        mbar_init(&b->k_empty[i], tiles);
        mbar_init(&b->v_empty[i], tiles);
        mbar_init(&b->s_full[i], 1);
        mbar_init(&b->p_full[i][0], kSoftWarps / 2);
        mbar_init(&b->p_full[i][1], kSoftWarps / 2);
        mbar_init(&b->o_full[i], 1);
        mbar_init(&b->fin[i], 1);
    }
    mbar_init(&b->go, kSoftWarps / 2);
    fence_mbar_init();
}

__device__ __forceinline__ void tear_down(Bars* b) {
    uint64_t* bar = reinterpret_cast<uint64_t*>(b);
    for (int i = 0; i < (int)(sizeof(Bars) / sizeof(uint64_t)); ++i) {
        asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar + i)) : "memory");
    }
}

// All roles of the block, each in code of its own: what was written before is there for all.
__device__ __forceinline__ void meet() {
    __syncwarp();
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
    tc_fence_after();
}

// The pieces of a block's stretch: steps u0 .. u1 - 1 of an item, and the piece's number.
template <typename Work>
__device__ __forceinline__ void walk(const CacheAttention& p, const Stretch& all, Work work) {
    int request = all.request, turn = 0;
    int64_t first = all.first;
    for (int64_t at = all.begin; at < all.end;) {
        const Item it = item_at(p, at, request, first);
        const int64_t last = it.begin + it.nominal < all.end ? it.begin + it.nominal : all.end;
        const int u0 = (int)min(at - it.begin, (int64_t)it.steps);
        const int u1 = (int)min(last - it.begin, (int64_t)it.steps);
        at = last;
        if (u0 < u1) work(it, u0, u1, turn++);   // (else steps that the tile does not need)
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cache_prompt_kernel(CacheAttention p) {
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                             ~(uintptr_t)1023);
    Shared* s = reinterpret_cast<Shared*>(sm + Layout<D>::scales);
    const int w = threadIdx.x >> 5;
    let_follow();
    // (the earliest any CTA can report a wait is seconds away)
    if (p.clears && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    const Stretch all = stretch_of<kThreads>(p, blockIdx.x, gridDim.x);
    if (all.request < 0) return;
    if (w == kIssueWarp) {
        if ((threadIdx.x & 31) == 0) s->abort = 0;
        __syncwarp();
        tmem_alloc(&s->tmem, 512);
        tmem_relinquish();
    }
    // Every role walks the block's pieces by itself, and all meet before and after each.  (One
    // walk for all would leave every role with the registers of the launch.)
    if (w < kSoftWarps) {
        take_registers<kSoftRegs>();
        walk(p, all, [&](const Item& it, int u0, int u1, int turn) {
            const float factor = stage_query<D>(p, it, sm);
            meet();
            const int t = threadIdx.x >> 7;
            float* part = u0 == 0 && u1 == it.steps
                              ? nullptr
                              : part_of(p, blockIdx.x, it.begin <= all.begin, D);
            if (t == 0 || it.rows > kRows) {
                soften<D>(p, it, s, &s->bars[turn & 1], u0, u1 - u0, t, factor, part);
            }
            meet();
        });
    } else if (w < kIssueWarp) {
        give_registers<kFillRegs>();
        walk(p, all, [&](const Item& it, int u0, int u1, int turn) {
            meet();
            const int high = it.hidden + (it.row0 + it.rows - 1) / p.group;
            fill<D>(p, it, s, &s->bars[turn & 1], sm, u0, u1 - u0, high);
            meet();
        });
    } else {
        give_registers<kIssueRegs>();
        walk(p, all, [&](const Item& it, int u0, int u1, int turn) {
            const int tiles = it.rows > kRows ? 2 : 1;
            Bars* b = &s->bars[turn & 1];
            if (threadIdx.x == 32 * kIssueWarp) {
                if (turn > 1) tear_down(b);  // (of the piece before the last: long over)
                set_up(b, tiles);
            }
            meet();
            if (w - kIssueWarp < tiles) {
                issue<D>(p, s, b, smem_u32(sm), u1 - u0, w - kIssueWarp);
            }
            meet();
        });
    }
    if (w == kIssueWarp) tmem_dealloc(s->tmem, 512);
}

// Joins the parts of the item that ends among block blockIdx.x's steps and began before them;
// kJoinRows of its rows.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) cache_prompt_join_kernel(CacheAttention p) {
    __shared__ float tops[kJoinRows], by[kJoinRows];
    let_follow();
    const Stretch all = stretch_of<kJoinThreads>(p, blockIdx.x, gridDim.x);
    wait_before();
    if (all.request < 0) return;
    int request = all.request;
    int64_t first = all.first;
    const Item it = item_at(p, all.begin, request, first);
    const int64_t b0 = it.begin / all.per, b1 = (it.begin + it.steps - 1) / all.per;
    // (an item whose steps all lie in one block is whole there)
    if (it.begin >= all.begin || it.begin + it.nominal > all.end || b0 == b1) return;
    const int r0 = blockIdx.y * kJoinRows;
    const int rows = it.rows - r0 < kJoinRows ? it.rows - r0 : kJoinRows;
    auto part = [&](int64_t b) { return part_of(p, b, it.begin <= b * all.per, D); };
    const int n = threadIdx.x;
    if (n < rows) {
        float top = kNone, l = 0.0f;
        for (int64_t b = b0; b <= b1; ++b) top = fmaxf(top, part(b)[2 * kRows * D + r0 + n]);
        const float ref = top == kNone ? 0.0f : top;
        for (int64_t b = b0; b <= b1; ++b) {
            const float* x = part(b) + 2 * kRows * D + r0 + n;
            l = fmaf(exp2_of(x[0] - ref), x[2 * kRows], l);
        }
        tops[n] = ref;
        by[n] = l == 0.0f ? 0.0f : 1.0f / l;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * D / 4; i += kJoinThreads) {
        const int r = 4 * i / D, c = 4 * i - r * D;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int64_t b = b0; b <= b1; ++b) {
            const float* x = part(b);
            const float f = exp2_of(x[2 * kRows * D + r0 + r] - tops[r]);
            const float4 v = *reinterpret_cast<const float4*>(x + (r0 + r) * D + c);
            y.x = fmaf(f, v.x, y.x);
            y.y = fmaf(f, v.y, y.y);
            y.z = fmaf(f, v.z, y.z);
            y.w = fmaf(f, v.w, y.w);
        }
        const int flat = it.row0 + r0 + r, j = flat / p.group;
        const int64_t to = ((it.token0 + j) * (p.heads * p.group) + it.head * p.group + flat -
                            j * p.group) * D + c;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x * by[r], y.y * by[r]);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(y.z * by[r], y.w * by[r]);
        const bool none = by[r] == 0.0f;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + to) =
            make_uint2(none ? 0u : *reinterpret_cast<const uint32_t*>(&lo),
                       none ? 0u : *reinterpret_cast<const uint32_t*>(&hi));
    }
}

template <int D>
cudaError_t launch_dim(const CacheAttention& p, int sms, cudaStream_t stream) {
    cudaError_t err = cudaFuncSetAttribute(
        cache_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::bytes);
    if (err != cudaSuccess) return err;
    cache_prompt_kernel<D><<<sms, kThreads, Layout<D>::bytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool cache_prompt_takes(int32_t d, int dtype) { return dtype == 1 && (d == 64 || d == 128); }

size_t cache_prompt_room(int32_t d, int sms) {
    return (size_t)sms * 2 * (2 * kRows) * (d + 2) * sizeof(float);
}

cudaError_t launch_cache_prompt(const CacheAttention& p, int sms, cudaStream_t stream) {
    return p.d == 64 ? launch_dim<64>(p, sms, stream) : launch_dim<128>(p, sms, stream);
}

cudaError_t launch_cache_prompt_join(const CacheAttention& p, int sms, cudaStream_t stream) {
    return launch_follower(p.d == 64 ? cache_prompt_join_kernel<64> : cache_prompt_join_kernel<128>,
                           dim3(sms, 2 * kRows / kJoinRows), dim3(kJoinThreads), 0, stream, p);
}

}  // namespace kda
