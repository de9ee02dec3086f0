// kda_lin_sm103.cu -- decayed linear attention on the tensor cores (bf16,
// dx = dz = 128): tcgen05 products on TMA tiles, accumulators in TMEM.
//
// One CTA walks one segment of one (sequence, head) in chunks of 128 tokens.
// With a = e^g and the chunk's rows i, j, per chunk (forward in time):
//     P   = X Y^T                                      (128 x 128 x 128)
//     P'  = mask(P) a^{i-j} kv_scale, bf16
//     O   = a^{i+1} X S + P' Z                         (2 products)
//     S'  = a^c S + (w Y)^T Z,  w_j = a^{c-1-j} kv_scale
// The state stays in fp32 registers; X S takes a bf16 copy of it (one
// rounding, as P' takes one).  w Y is split into three bf16 parts (8 + 8 + 8
// bits), so that the state keeps fp32 sums of exact products: three products
// on a tensor core that otherwise waits for memory.
//
// What bounds it: the rows are read and written once (131 KB a chunk), and with
// all SMs at work a chunk of 128 tokens takes 3.2 - 3.6 us an SM, 79 - 83 % of a plain copy's
// rate on a ragged batch of 109,824 tokens and 64 heads (1,305 - 1,372 us).  A CTA alone on
// its memory still takes 2.95 us: the chain S -> X S -> state, and about 480 KB of
// shared memory that the products and the copies move a chunk (1.85 us at 128
// bytes a cycle).  The tensor core itself is busy for 42 %.  A fixed 10 us a CTA
// (TMEM, tables, the first tiles, the last outputs) is what short sequences pay.
//
// Few pairs of sequence and head leave SMs idle.  Then sequences are cut into
// segments: one kernel forms the state that each segment adds (Y and Z alone, the
// sums in TMEM over four chunks at a time: 1.6 us a chunk), a scan carries them
// on, and the pass starts each segment from its state.  One sequence of 4,096 tokens,
// 32 heads: 65 us (about 22 states, 6 scan, 37 pass, one after another; each kernel is brought on
// while the one before ends) where whole sequences took 108.
//
// Roles (28 warps): 0-7 turn P into P' and write the outputs (thread = token;
// each half takes half of the columns), 8-15 carry the state (thread = row of
// S; half of the columns each), 16-23 split w Y (half of the tokens each), 24
// issues the TMA loads, 25 the products, 26 the TMA stores.
#include "kda_lin.h"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <limits.h>
#include <string.h>

#include "kda_follow.cuh"
#include "kda_lin.cuh"
#include "kda_packed.cuh"
#include "sm103_ptx.cuh"

namespace kda {
namespace {

using namespace sm103;

constexpr int C = 128;                   // tokens per chunk = rows of a tile
constexpr int D = 128;                   // dx = dz
constexpr int THREADS = 896;             // the pass
constexpr int STATE_THREADS = 576;       // the segment states: 16 warps, and 16 and 17 to issue
// Registers: 896 threads start with 72 each.  The warps that issue and those
// that split give some up for the 8 that hold the state:
// 128 (72 + 72 + 96 + 96 + 64 + 64 + 40) = 896 x 72.
constexpr int REGS = 72, REGS_STATE = 96, REGS_SPLIT = 64, REGS_ISSUE = 40;
static_assert(128 * (2 * REGS + 2 * REGS_STATE + 2 * REGS_SPLIT + REGS_ISSUE) <= THREADS * REGS,
              "register split");
constexpr uint32_t HALF = C * 128;       // a tile's 64 columns: 128 rows of 128 bytes
constexpr uint32_t TILE = 2 * HALF;
constexpr int STAGES = 2;                // the pass: X, Y, Z per stage
constexpr int STATE_STAGES = 3;          // the segment states: Y, Z per stage
static_assert(D * D * 4 <= 3 * TILE, "the state before a segment fits stage 1");
constexpr uint32_t SM_S = STAGES * 3 * TILE;             // bf16 copy of the state
constexpr uint32_t SM_TAB = SM_S + TILE;
static_assert(SM_S >= STATE_STAGES * 2 * TILE, "the states' stages end before the copy");
constexpr uint32_t SMEM = SM_TAB + 2048 + 1024;          // tables, alignment
static_assert(SMEM <= 232448, "more shared memory than a CTA may have");

// All 512 columns of TMEM are allocated, so that their base is 0 and addresses
// are constants.
// TMEM columns of the pass.  P' (bf16 pairs) takes the first 16 of each 32
// columns of P.
constexpr uint32_t TC_P = 0;
constexpr uint32_t TC_O = 128;           // X S, scaled in place, then + P' Z
constexpr uint32_t TC_U = 256;           // (w Y)^T Z
constexpr uint32_t TC_W = 384;           // w Y of 32 tokens: two buffers of three parts of 16
// and of the segment states
constexpr uint32_t TS_U = 0;
constexpr uint32_t TS_W = 128;           // two buffers of three parts of 64 columns

// The tables: weights of a whole chunk's tokens in the state, then the powers of the
// decay, then the barriers.  split_w reads a short chunk's weights from the middle of
// the first on, up to C - 1 entries past its end: into the second, never past it.
constexpr int POWERS = C + 4;
static_assert(C - 1 <= POWERS, "reads past the weights stay in the tables");
static_assert((C + POWERS) * 4 + 320 <= 2048, "tables and barriers");

struct Args {
    CUtensorMap x, y, z, out;
    CUtensorMap init, segs, last;  // states: the initial, between the segments, the final ones
    LinPass p;
};

// Up to three passes of the same sizes in one launch: the gradients of q, k and v
// need nothing of each other.
struct Jobs {
    Args a[3];
    int n;
    int first;                     // the call's first kernel: it clears the status word
};

struct Bars {
    uint64_t full[STATE_STAGES];   // tiles of a stage are there
    uint64_t empty[STATE_STAGES];  // products on a stage are done
    uint64_t qk, o1, o2, u;        // P / X S / P' Z / (w Y)^T Z done
    uint64_t p, s, o1s, od;        // P' / S copy / X S scaled / outputs written
    uint64_t xfree[2];             // the outputs have left the stage's X tile
    uint64_t w[2], wfree[2];       // w Y of a buffer written, read
    uint64_t init, begun, end;     // the state before the segment there / taken over; after it written
    uint64_t joined;               // the sums so far have been taken out of TMEM
    uint64_t fin;
    uint32_t tmem;
    volatile int abort;
};

static_assert(sizeof(Bars) <= 320, "barriers");

// 3-D tiled store of one box from shared memory, in this thread's bulk group.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int c0,
                                             int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], "
                 "[%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until the bulk stores of this thread have read their shared memory (READ), or
// are done.
template <bool READ>
__device__ __forceinline__ void bulk_wait() {
    if (READ) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    } else {
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
}

// Bounded wait that sleeps in the barrier, up to 20 us at a time, instead of
// polling: polls would take issue slots from the warps that work.  False when
// the CTA gives up, or after WAIT_TRIES (some 10 s if every one sleeps its time
// out; a wait of these kernels is over in microseconds).
constexpr uint32_t WAIT_TRIES = 1u << 19;

__device__ __forceinline__ bool sleep_wait(Bars* b, uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_u32(bar);
    for (uint32_t i = 0; i < WAIT_TRIES; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(at), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
        if (b->abort) return false;
    }
    return false;
}

__device__ __forceinline__ void give_up(const LinPass& p, Bars* b, int site) {
    atomicCAS(p.status, 0, site);
    b->abort = 1;
}

// One thread's bounded wait; on a timeout every role of the CTA leaves its loop.
__device__ __forceinline__ bool wait1(Bars* b, uint64_t* bar, uint32_t parity, const LinPass& p,
                                      int site) {
    if (sleep_wait(b, bar, parity)) return true;
    give_up(p, b, site);
    return false;
}

// The same for a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool wait_warp(Bars* b, uint64_t* bar, uint32_t parity,
                                          const LinPass& p, int site) {
    const bool ok = sleep_wait(b, bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    give_up(p, b, site);
    return false;
}

// One arrival for the calling warp, behind what all of its lanes did.
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The upper halves of a and b.
__device__ __forceinline__ uint32_t cut(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

__device__ __forceinline__ float upper(float a) {
    return __uint_as_float(__float_as_uint(a) & 0xffff0000u);
}

// Low words of the shared-memory descriptors of an operand tile; the steps of a
// product add to the address in them.  One thread issues every product, so each
// is kept to a few instructions.  The high word (128-byte swizzle, 1024 bytes
// between groups of 8 rows) is the same for all.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
// K-major: rows of 64 channels; k-step kk covers 16 channels.
__device__ __forceinline__ uint32_t tile_k(uint32_t tile) { return tile >> 4 | 1u << 16; }
__device__ __forceinline__ constexpr uint32_t step_k(int kk) {
    return ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
}
// MN-major: rows are the summed index; k-step kk covers 16 rows.
__device__ __forceinline__ uint32_t tile_mn(uint32_t tile) { return tile >> 4 | (HALF >> 4) << 16; }
__device__ __forceinline__ constexpr uint32_t step_mn(int kk) { return kk * 2048 >> 4; }

// D (+)= A B of 128 x 128 x 16: A in shared memory, or in TMEM.  The whole warp
// calls it, so that the operands stay in uniform registers, and one lane (always
// the same) issues.
template <bool ADD>
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %4};\n\t"
        "mov.b64 b, {%2, %4};\n\tsetp.ne.b32 p, %5, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(DESC_HI), "n"(ADD ? 1 : 0)
        : "memory");
}
template <bool ADD>
__device__ __forceinline__ void product_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %4};\n\t"
        "setp.ne.b32 p, %5, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(DESC_HI), "n"(ADD ? 1 : 0)
        : "memory");
}

// Arrives once every product issued so far is done (the same lane).
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::
            "r"(smem_u32(bar))
        : "memory");
}

// 16 TMEM lanes x 16 columns: register j of lane l holds row l / 4 + 8 (j & 1),
// column 4 (j / 2) + l % 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

// Four 8 x 8 matrices, transposed: register k of lane l holds rows 2 (l % 4)
// and + 1, column l / 4 of matrix k, whose row i lane 8 k + i points to.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// w Y of this warp's 32 rows of S (TMEM lanes) for 32 tokens, split into three
// bf16 parts: bits cut off twice, the rest rounded, so that the parts add up
// to the fp32 product within 2^-24.  The tile is read transposed, 8 x 8 values
// at a time, into the layout that TMEM takes 16 lanes at a time.  w: the weight
// of token 0 of the chunk; rows past its end (another sequence's, maybe not
// finite) count as zero, and their weights are read from the table behind.
__device__ __forceinline__ void split_w(uint32_t y, int quad, int tok0, const float* w, float f,
                                        int len, uint32_t hi, uint32_t mid, uint32_t lo) {
    const int lane = threadIdx.x & 31, row = lane & 7, mat = lane >> 3;
    const int t0 = tok0 + 2 * (lane & 3);
    uint64_t ws[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)   // (single loads: a short chunk's table starts anywhere)
        ws[j] = mul2(two(w[t0 + 8 * j], w[t0 + 8 * j + 1]), two(f, f));
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const int chunk = (quad & 1) * 4 + 2 * half + (mat & 1);
        const uint32_t at = y + (quad >> 1) * HALF + (tok0 + 8 * (mat >> 1) + row) * 128 +
                            ((chunk ^ row) << 4);
        uint32_t h[8], m[8], l[8];
        ldmatrix_x4_trans(at, h);
        ldmatrix_x4_trans(at + 16 * 128, h + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint64_t x = mul2(two(low(h[j]), high(h[j])), ws[j >> 1]);
            float x0, x1;
            apart(x, x0, x1);
            if (len < C) {
                if (t0 + 8 * (j >> 1) >= len) x0 = 0.0f;
                if (t0 + 8 * (j >> 1) + 1 >= len) x1 = 0.0f;
            }
            h[j] = cut(x0, x1);
            x = sub2(two(x0, x1), two(upper(x0), upper(x1)));
            apart(x, x0, x1);
            m[j] = cut(x0, x1);
            l[j] = pack(sub2(x, two(upper(x0), upper(x1))));
        }
        const uint32_t lanes = (uint32_t)half << 20;   // lane 16 of the warp's 32
        tmem_st_16x128b_x4(hi + lanes, h);
        tmem_st_16x128b_x4(mid + lanes, m);
        tmem_st_16x128b_x4(lo + lanes, l);
    }
}

// What ordinary stores write to shared memory is made visible to TMA and the
// tensor core by a proxy fence of the warp that issues those, behind the barrier
// that the writers arrived on: in every writer, where it waits for the writer's
// own stores, the fence took some 900 cycles of each hand-over.

// Rows len .. 127 of a Z tile to zero: they meet zeros of P' and w Y, and may
// hold another sequence's values, which need not be finite.
__device__ __forceinline__ void zero_rows(uint8_t* z, int len, int tid, int threads) {
    for (int i = tid; i < (C - len) * 16; i += threads) {
        const int row = len + (i >> 4), part = i & 15;
        *reinterpret_cast<uint4*>(z + (part >> 3) * HALF + row * 128 + (part & 7) * 16) =
            make_uint4(0, 0, 0, 0);
    }
}

__device__ __forceinline__ void load_tile(const CUtensorMap* map, uint8_t* dst, int h, int tok,
                                          uint64_t* bar) {
    tma_load_3d(dst, map, 0, h, tok, bar);
    tma_load_3d(dst + HALF, map, 64, h, tok, bar);
}

// What every CTA of both kernels starts with.
struct Cta {
    uint8_t* sm;
    Bars* b;
    float* wtab;    // weights of a whole chunk's tokens in the state
    float* lam;     // a^0 .. a^128
    lin::Segment sg;
    int h, chunks;
    bool rev;
    float g;
};

// The pass and the segment of this CTA (heads fastest, then the passes, then the
// segments).  Whole sequences come longest first, so that none starts late; of
// sequences cut in two the tails, and then the heads.
template <bool STATES>
__device__ __forceinline__ const Args* start(const Jobs& jobs, Cta& c) {
    // (the earliest any CTA can report a wait is seconds away)
    if (jobs.first && blockIdx.x == 0 && threadIdx.x == 0) *jobs.a[0].p.status = 0;
    extern __shared__ uint8_t smem_raw[];
    const int H = jobs.a[0].p.H, unit = blockIdx.x / H;
    const Args* args = &jobs.a[unit % jobs.n];
    const LinPass& p = args->p;
    c.sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~(uintptr_t)1023);
    c.wtab = reinterpret_cast<float*>(c.sm + SM_TAB);
    c.lam = c.wtab + C;
    c.b = reinterpret_cast<Bars*>(c.lam + POWERS);
    c.h = blockIdx.x % H;
    c.rev = p.reverse != 0;
    int index = unit / jobs.n;
    if (p.lead > 0 && STATES) {
        c.sg = lin::lead_segment(p.cu_seqlens, p.N, p.total_T, p.seg_len, p.reverse, p.lead,
                                 index % p.N, index / p.N);
        return c.sg.n >= 0 ? args : nullptr;
    }
    const bool tail = p.lead > 0 && index < p.N;
    if (p.lead > 0 && !tail) index -= p.N;
    if (p.cu_seqlens && p.N <= lin::RANKED && (p.lead > 0 || p.total_T < p.seg_len))
        index = lin::nth_longest(p.cu_seqlens, p.N, p.total_T, index);
    c.sg = p.lead > 0 ? lin::half_segment(p.cu_seqlens, p.N, p.total_T, p.seg_len, p.reverse,
                                          p.lead, index, tail)
                      : lin::find_segment(p.cu_seqlens, p.N, p.total_T, p.seg_len, p.reverse,
                                          index);
    return c.sg.n >= 0 ? args : nullptr;
}

// Token range of the pass's step i.
__device__ __forceinline__ int64_t chunk_start(const Cta& c, int i) {
    return c.sg.t0 + (int64_t)(c.rev ? c.chunks - 1 - i : i) * C;
}
__device__ __forceinline__ int chunk_len(const Cta& c, int64_t tok) {
    return (int)(c.sg.t1 - tok < C ? c.sg.t1 - tok : C);
}

// `issue`: the first of the issuing warps; `w_warps`: those that fill a buffer of w Y;
// `first`: the first loads, which one thread issues as soon as the barriers are there,
// under the tables and the allocation.
template <typename First>
__device__ __forceinline__ void set_up(const Args& args, Cta& c, int issue, int w_warps,
                                       First first) {
    const LinPass& p = args.p;
    const int tid = threadIdx.x;
    c.chunks = (int)((c.sg.t1 - c.sg.t0 + C - 1) / C);
    if (tid == 32 * issue) {
        Bars* b = c.b;
        for (int i = 0; i < STATE_STAGES; ++i) {
            mbar_init(&b->full[i], 1);
            mbar_init(&b->empty[i], 1);
        }
        uint64_t* one[] = {&b->init, &b->xfree[0], &b->xfree[1], &b->qk, &b->o1, &b->o2, &b->u, &b->wfree[0], &b->wfree[1], &b->fin};
        uint64_t* all[] = {&b->p, &b->s, &b->o1s, &b->od, &b->begun};
        for (uint64_t* x : one) mbar_init(x, 1);
        for (uint64_t* x : all) mbar_init(x, 8);   // warps
        for (uint64_t& x : b->w) mbar_init(&x, w_warps);
        mbar_init(&b->end, w_warps == 4 ? 8 : w_warps);   // the warps that hold a state
        mbar_init(&b->joined, w_warps);
        b->abort = 0;
        fence_mbar_init();
        fence_proxy_async();
        first();
    }
    if (tid >> 5 == issue + 1) {
        tmem_alloc(&c.b->tmem, 512);
        tmem_relinquish();
    }
    c.g = p.log_decay[c.h];
    if (tid <= C) {
        const float a = lin::decay_pow(c.g, tid);
        c.lam[tid] = a;
        if (p.reverse ? tid > 0 : tid < C) c.wtab[p.reverse ? tid - 1 : C - 1 - tid] = a * p.kv_scale;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

__device__ __forceinline__ void finish(const Cta& c, int issue) {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x >> 5 == issue + 1) tmem_dealloc(c.b->tmem, 512);
}

// ------------------------------------------------------------------ the pass
template <int N>
__device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The state before the segment, or null (zeros): the initial one, or the one that
// the scan left in the row of the segment before.
__device__ __forceinline__ const float* start_state(const LinPass& p, const Cta& c) {
    const int64_t rows = lin::seg_rows(p.total_T, p.seg_len);
    if (c.sg.j > 0) {
        if (c.sg.u + c.sg.j - 1 >= rows) return nullptr;   // only a malformed cu_seqlens
        return p.seg_states + ((c.sg.u + c.sg.j - 1) * (int64_t)p.H + c.h) * (int64_t)(D * D);
    }
    return p.state_in ? p.state_in + ((size_t)c.sg.n * p.H + c.h) * (size_t)(D * D) : nullptr;
}

// The state before the segment, where TMA brings it, and the first chunk.
__device__ __forceinline__ bool tma_start(const LinPass& p, const Cta& c) {
    return (c.sg.j > 0 || !p.state_in_turned) && start_state(p, c);
}

__device__ __forceinline__ void first_loads(const Args& args, const Cta& c) {
    const LinPass& p = args.p;
    Bars* b = c.b;
    if (c.chunks > 0) {
        const int tok = (int)chunk_start(c, 0);
        mbar_arrive_expect_tx(&b->full[0], 3 * TILE);
        load_tile(&args.y, c.sm + TILE, c.h, tok, &b->full[0]);
        load_tile(&args.x, c.sm, c.h, tok, &b->full[0]);
        load_tile(&args.z, c.sm + 2 * TILE, c.h, tok, &b->full[0]);
    }
    wait_before();             // the segments' states
    fence_proxy_async();
    if (tma_start(p, c)) {
        mbar_arrive_expect_tx(&b->init, D * D * 4);
        const CUtensorMap* map = c.sg.j > 0 ? &args.segs : &args.init;
        const int state = (int)(c.sg.j > 0 ? (c.sg.u + c.sg.j - 1) * p.H + c.h
                                           : (int64_t)c.sg.n * p.H + c.h);
        for (int q = 0; q < D / 32; ++q)
            tma_load_3d(c.sm + 3 * TILE + q * HALF, map, 32 * q, 0, state, &b->init);
    }
}

__device__ __forceinline__ void issue_loads(const Args& args, const Cta& c) {
    const LinPass& p = args.p;
    Bars* b = c.b;
    int issued = c.chunks > 0;
    for (int i = 1; i < c.chunks; ++i) {
        const int s = i & 1;
        // stage 1 holds the state first
        if (i == 1 && !wait1(b, &b->begun, 0, p, 317)) break;
        if (i >= STAGES && !wait1(b, &b->empty[s], ((i >> 1) - 1) & 1, p, 301)) break;
        uint8_t* st = c.sm + s * 3 * TILE;
        const int tok = (int)chunk_start(c, i);
        mbar_arrive_expect_tx(&b->full[s], 3 * TILE);
        load_tile(&args.y, st + TILE, c.h, tok, &b->full[s]);
        load_tile(&args.z, st + 2 * TILE, c.h, tok, &b->full[s]);
        // (the expected bytes are all announced, so a give-up here still loads X)
        if (i >= STAGES) wait1(b, &b->xfree[s], ((i >> 1) - 1) & 1, p, 315);
        load_tile(&args.x, st, c.h, tok, &b->full[s]);
        issued = i + 1;
    }
    // no copy outlives the CTA
    for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
        mbar_wait(&b->full[i & 1], (i >> 1) & 1, nullptr);
    if (tma_start(p, c)) mbar_wait(&b->init, 0, nullptr);
}

// Whether the CTA writes a final state.
__device__ __forceinline__ bool hands_on(const LinPass& p, const Cta& c) {
    return p.state_out && c.sg.j + 1 == c.sg.count;
}

// Four values of row r of a state to where store_states takes them from.
__device__ __forceinline__ void store_state(uint8_t* tiles, int r, int col, const float* v) {
    *reinterpret_cast<float4*>(tiles + (col >> 5) * HALF + sw128(r, (col & 31) * 4)) =
        make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_states(const CUtensorMap* map, const uint8_t* tiles,
                                             int state) {
    fence_proxy_async();
    for (int q = 0; q < D / 32; ++q) tma_store_3d(map, tiles + q * HALF, 32 * q, 0, state);
    bulk_commit();
}

// The outputs of whole chunks, from the X tiles to memory, and the final state.
__device__ __forceinline__ void issue_stores(const Args& args, const Cta& c) {
    const LinPass& p = args.p;
    Bars* b = c.b;
    for (int i = 0; i < c.chunks; ++i) {
        if (!wait1(b, &b->od, i & 1, p, 316)) break;
        const int64_t tok = chunk_start(c, i);
        if (chunk_len(c, tok) == C) {
            const uint8_t* tile = c.sm + (i & 1) * 3 * TILE;
            fence_proxy_async();
            tma_store_3d(&args.out, tile, 0, c.h, (int)tok);
            tma_store_3d(&args.out, tile + HALF, 64, c.h, (int)tok);
            bulk_commit();
            bulk_wait<true>();
        }
        mbar_arrive(&b->xfree[i & 1]);
    }
    if (hands_on(p, c) && !b->abort && wait1(b, &b->end, 0, p, 318))
        store_states(&args.last, c.sm + TILE, c.sg.n * p.H + c.h);
    bulk_wait<false>();
}

// The products of all chunks, in the order in which the tensor core runs them.
// P of the next chunk comes last: it fills the time that the state takes.
__device__ __forceinline__ void issue_products(const LinPass& p, const Cta& c) {
    Bars* b = c.b;
    constexpr uint32_t id_kk = idesc_bf16(D, D, 0, 0), id_km = idesc_bf16(D, D, 0, 1);
    const uint32_t base = smem_u32(c.sm), state = tile_mn(base + SM_S);
    const int n = c.chunks;
    for (int i = -1; i < n; ++i) {
        const uint32_t ph = i & 1;
        if (i >= 0) {
            const uint32_t tile = base + ph * 3 * TILE, x = tile_k(tile);
            const uint32_t z = tile_mn(tile + 2 * TILE);
            if (!wait_warp(b, &b->s, ph, p, 304)) break;
            if (i > 0 && !wait_warp(b, &b->od, ph ^ 1, p, 314)) break;
            fence_proxy_async();   // the state's copy
            tc_fence_after();
            product<false>(TC_O, x, state, id_km);
#pragma unroll
            for (int kk = 1; kk < 8; ++kk)
                product<true>(TC_O, x + step_k(kk), state + step_mn(kk), id_km);
            commit(&b->o1);
            // a short chunk's z rows past its end are zeroed before P' is handed over
            if (chunk_len(c, chunk_start(c, i)) < C) {
                if (!wait_warp(b, &b->p, ph, p, 306)) break;
                fence_proxy_async();
            }
            bool ok = true;
#pragma unroll
            for (int g = 0; g < 4; ++g) {     // w Y of 32 tokens each
                const int buf = g & 1;
                if (g == 2) {
                    ok = wait_warp(b, &b->p, ph, p, 307) && wait_warp(b, &b->o1s, ph, p, 308);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        product_ta<true>(TC_O, TC_P + 32 * (kk >> 1) + 8 * (kk & 1),
                                         z + step_mn(kk), id_km);
                    commit(&b->o2);
                }
                if (!(ok = wait_warp(b, &b->w[buf], g >> 1, p, 305))) break;
                tc_fence_after();
                const uint32_t w = TC_W + 48 * buf;
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const uint32_t zk = z + step_mn(2 * g + kk);
                    if (g == 0 && kk == 0) {
                        product_ta<false>(TC_U, w + 32, zk, id_km);
                    } else {
                        product_ta<true>(TC_U, w + 32 + 8 * kk, zk, id_km);
                    }
                    product_ta<true>(TC_U, w + 16 + 8 * kk, zk, id_km);
                    product_ta<true>(TC_U, w + 8 * kk, zk, id_km);
                }
                commit(&b->wfree[buf]);
            }
            if (!ok) break;
            commit(&b->u);
            commit(&b->empty[ph]);
        }
        if (i + 1 < n) {
            const uint32_t next = base + (ph ^ 1) * 3 * TILE, x = tile_k(next);
            const uint32_t y = tile_k(next + TILE);
            if (!wait_warp(b, &b->full[ph ^ 1], ((i + 1) >> 1) & 1, p, 302)) break;
            if (i >= 0 && !wait_warp(b, &b->o2, ph, p, 303)) break;   // P' has been read
            tc_fence_after();
            product<false>(TC_P, x, y, id_kk);
#pragma unroll
            for (int kk = 1; kk < 8; ++kk)
                product<true>(TC_P, x + step_k(kk), y + step_k(kk), id_kk);
            commit(&b->qk);
        }
    }
    commit(&b->fin);
    mbar_wait(&b->fin, 0, nullptr);   // no product outlives the CTA
}

// 32 columns of P, as bf16 pairs, column s weighted by 2^{g2 |t - s| + c}.  The
// weights are formed on the spot, as 2^{base + slope s}: a table in shared memory
// would wait for the products' own reads of it.  Their error, 2^-22 and that of the
// exponent (at most 31 |g2| 2^-24: 2^-20 for decays down to e^-0.35 a token, up to 2.4e-4, a
// sixteenth of the bf16 rounding that follows, at the strongest that counts, g2 = -128), comes
// before the rounding to bf16.  MASKED: only columns first .. last of the block count.
template <bool MASKED>
__device__ __forceinline__ void weigh(uint32_t col, float base, float slope, int first, int last) {
    uint32_t r[2][16], w[16];
    tmem_ld16(col, r[0]);
    tmem_ld16(col + 16, r[1]);
    tmem_wait_ld();
    const bool none = last < first;
    const uint32_t from = none ? 64 : first, span = none ? 0 : last - first;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int s = 2 * j;
        uint64_t v = mul2(two(r[j >> 3][s & 15], r[j >> 3][(s & 15) + 1]),
                          two(exp2_approx(fmaf(slope, (float)s, base)),
                              exp2_approx(fmaf(slope, (float)(s + 1), base))));
        if (MASKED) {
            float v0, v1;
            apart(v, v0, v1);
            if (s - from > span) v0 = 0.0f;
            if (s + 1 - from > span) v1 = 0.0f;
            v = two(v0, v1);
        }
        w[j] = pack(v);
    }
    tmem_st16(col, w);
}

// Warps 0-7: P' (columns 32 q with q even or odd) and the outputs (columns 64 grp on).
__device__ __forceinline__ void outputs(const LinPass& p, const Cta& c, uint32_t lanes) {
    Bars* b = c.b;
    const int t = threadIdx.x & 127, quad = (threadIdx.x >> 5) & 3, grp = threadIdx.x >> 7;
    // The exponent of a weight: slope s + base.  log2 a is kept above -128, where a
    // distance of one already weighs nothing (2^-128 is no fp32 of full precision),
    // so that a distance of zero weighs 1 under every decay.  The pass's two scales
    // go into the weights and, once more, into X S; their sign into the outputs.
    const float g2 = c.g < -88.0f ? -128.0f : c.g * 1.44269504f, slope = c.rev ? g2 : -g2;
    const float scale = p.out_scale * p.kv_scale;
    const float c2 = log2f(fabsf(scale));
    const uint32_t flip = scale < 0.0f ? 0x80008000u : 0u;
    const float m = scale < 0.0f ? -p.out_scale : p.out_scale;
    for (int i = 0; i < c.chunks; ++i) {
        const uint32_t ph = i & 1;
        const int64_t tok = chunk_start(c, i);
        const int len = chunk_len(c, tok);
        if (len < C) {
            if (!wait_warp(b, &b->full[i & 1], (i >> 1) & 1, p, 310)) break;
            zero_rows(c.sm + (i & 1) * 3 * TILE + 2 * TILE, len, threadIdx.x, 256);
        }
        if (!wait_warp(b, &b->qk, ph, p, 311)) break;
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const int q = 2 * k + grp;
            const uint32_t col = lanes + TC_P + 32 * q;
            const int tq = t - 32 * q;
            const float base = fmaf(-slope, (float)tq, c2);
            if ((c.rev ? q > quad : q < quad) && len == C) {
                weigh<false>(col, base, slope, 0, 31);
            } else if (c.rev ? q >= quad : q <= quad) {
                const int end = len - 32 * q - 1;
                weigh<true>(col, base, slope, c.rev ? max(tq, 0) : 0, c.rev ? end : min(tq, end));
            } else {
                const uint32_t zero[16] = {};
                tmem_st16(col, zero);
            }
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&b->p);

        const float f = t < len ? m * c.lam[c.rev ? len - 1 - t : t + 1] : 0.0f;
        const uint32_t o = lanes + TC_O + 64 * grp;
        if (!wait_warp(b, &b->o1, ph, p, 312)) break;
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < 4; q += 2) {
            uint32_t r[2][16];
            tmem_ld16(o + 16 * q, r[0]);
            tmem_ld16(o + 16 * q + 16, r[1]);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                float a, e;
                apart(mul2(two(r[j >> 4][j & 15], r[j >> 4][(j & 15) + 1]), two(f, f)), a, e);
                r[j >> 4][j & 15] = __float_as_uint(a);
                r[j >> 4][(j & 15) + 1] = __float_as_uint(e);
            }
            tmem_st16(o + 16 * q, r[0]);
            tmem_st16(o + 16 * q + 16, r[1]);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&b->o1s);

        // The outputs of a whole chunk leave through the X tile, which both
        // products that read it are done with, as one TMA store: a row per thread
        // written straight to memory would send 32 pieces of lines per warp store.
        uint8_t* tile = c.sm + (i & 1) * 3 * TILE + grp * HALF;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) +
                             ((size_t)(tok + t) * p.H + c.h) * D + 64 * grp;
        if (!wait_warp(b, &b->o2, ph, p, 313)) break;
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < 4; q += 2) {
            uint32_t r[2][16];
            tmem_ld16(o + 16 * q, r[0]);
            tmem_ld16(o + 16 * q + 16, r[1]);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = 8 * e + 2 * j;
                    w[j] = pack(__uint_as_float(r[k >> 4][k & 15]),
                                __uint_as_float(r[k >> 4][(k & 15) + 1])) ^ flip;
                }
                const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
                if (len == C) {
                    *reinterpret_cast<uint4*>(tile + sw128(t, 16 * (2 * q + e))) = v;
                } else if (t < len) {
                    reinterpret_cast<uint4*>(out + 16 * q)[e] = v;
                }
            }
        }
        tc_fence_before();
        arrive_warp(&b->od);
    }
}

// Warps 16-23: w Y of the chunks' tokens 32 grp on and 64 + 32 grp on, into the
// group's buffer.
__device__ __forceinline__ void weights(const LinPass& p, const Cta& c, uint32_t lanes) {
    Bars* b = c.b;
    const int quad = (threadIdx.x >> 5) & 3, grp = (threadIdx.x >> 7) & 1;
    const uint32_t w = lanes + TC_W + 48 * grp;
    bool ok = true;
    for (int i = 0; ok && i < c.chunks; ++i) {
        const uint32_t ph = i & 1;
        const int len = chunk_len(c, chunk_start(c, i));
        if (!wait_warp(b, &b->full[ph], (i >> 1) & 1, p, 320)) break;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            if ((half || i > 0) && !(ok = wait_warp(b, &b->wfree[grp], half ^ 1, p, 321))) break;
            tc_fence_after();
            split_w(smem_u32(c.sm) + ph * 3 * TILE + TILE, quad, 64 * half + 32 * grp,
                    c.wtab + (c.rev ? 0 : C - len), 1.0f, len, w, w + 16, w + 32);
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&b->w[grp]);
        }
    }
}

// Warps 8-15: the state (row r, columns 64 grp on).
__device__ __forceinline__ void states(const LinPass& p, const Cta& c, uint32_t lanes) {
    Bars* b = c.b;
    constexpr int W = D / 2;
    const int r = threadIdx.x & 127, grp = (threadIdx.x >> 7) & 1;
    float S[W];
#pragma unroll
    for (int j = 0; j < W; ++j) S[j] = 0.0f;
    bool ok = true;
    const float* start = start_state(p, c);
    if (start && (c.sg.j > 0 || !p.state_in_turned)) {
        // it comes into stage 1, 32 columns a tile, swizzled as the operands are
        ok = wait_warp(b, &b->init, 0, p, 323);
        const uint8_t* tile = c.sm + 3 * TILE + 2 * grp * HALF;
#pragma unroll
        for (int j = 0; j < W; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(tile + (j >> 5) * HALF +
                                                              sw128(r, (j & 31) * 4));
            S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
        }
    } else if (start) {
#pragma unroll
        for (int j = 0; j < W; ++j) S[j] = start[(size_t)(W * grp + j) * D + r];
    }
    arrive_warp(&b->begun);   // stage 1 is free
    uint8_t* copy = c.sm + SM_S + grp * HALF;
    for (int i = 0; ok && i <= c.chunks; ++i) {
        if (i > 0) {
            if (!(ok = wait_warp(b, &b->u, (i - 1) & 1, p, 322))) break;
            tc_fence_after();
            const float f = c.lam[chunk_len(c, chunk_start(c, i - 1))];
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
                uint32_t v[2][16];
                tmem_ld16(lanes + TC_U + 64 * grp + 16 * q, v[0]);
                tmem_ld16(lanes + TC_U + 64 * grp + 16 * q + 16, v[1]);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    apart(fma2(two(f, f), two(S[16 * q + j], S[16 * q + j + 1]),
                               two(v[j >> 4][j & 15], v[j >> 4][(j & 15) + 1])),
                          S[16 * q + j], S[16 * q + j + 1]);
            }
            tc_fence_before();
        }
        if (i == c.chunks) break;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            uint4 v;
            v.x = pack(S[8 * q], S[8 * q + 1]);
            v.y = pack(S[8 * q + 2], S[8 * q + 3]);
            v.z = pack(S[8 * q + 4], S[8 * q + 5]);
            v.w = pack(S[8 * q + 6], S[8 * q + 7]);
            *reinterpret_cast<uint4*>(copy + sw128(r, q * 16)) = v;
        }
        arrive_warp(&b->s);
    }
    if (ok && hands_on(p, c)) {
        // through the Y and Z tiles of stage 0, which nothing reads any more
#pragma unroll
        for (int j = 0; j < W; j += 4) store_state(c.sm + TILE, r, W * grp + j, &S[j]);
        arrive_warp(&b->end);
    }
}

__global__ void __launch_bounds__(THREADS, 1)
lin_pass_tc_kernel(const __grid_constant__ Jobs jobs) {
    Cta c;
    const Args* job = start<false>(jobs, c);
    if (!job) return;
    const Args& args = *job;
    const LinPass& p = args.p;
    set_up(args, c, 24, 4, [&] { first_loads(args, c); });
    const int warp = threadIdx.x >> 5;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's 32 TMEM lanes
    if (warp < 8) {
        outputs(p, c, lanes);
    } else if (warp < 16) {
        take_registers<REGS_STATE>();
        states(p, c, lanes);
    } else if (warp < 24) {
        give_registers<REGS_SPLIT>();
        weights(p, c, lanes);
    } else {
        give_registers<REGS_ISSUE>();
        if (warp == 25) {
            issue_products(p, c);
        } else if ((threadIdx.x & 31) == 0) {
            if (warp == 24) issue_loads(args, c);
            if (warp == 26) issue_stores(args, c);
        }
    }
    finish(c, 24);
}

// ------------------------------------------------- the state a segment adds
// sum_j a^{tokens from j to the segment's end} kv_scale y_j z_j^T, accumulated in TMEM:
// the weights are taken to the segment's end at once.  Sixteen warps split w Y
// into one of two buffers while the products read the other.
//
// The tensor core cuts its sums off to fp32 (it does not round them), always
// towards zero: over 256 chunks of one sign a state came out 7.7e-5 too small.  So
// JOIN chunks at most are added up there, and the splitting warps, which hold 32
// columns of the state each, add those sums up in registers.  64K prompt of 96 heads
// without joins, and joining every 8, 4, 2 chunks: 1,395, 1,409, 1,408, 1,413 us; 4K of
// 32 heads: 63.9, 63.5, 63.6, 64.2.
constexpr int JOIN = 4;

__global__ void __launch_bounds__(STATE_THREADS, 1)
lin_states_tc_kernel(const __grid_constant__ Jobs jobs) {
    Cta c;
    let_follow();
    const Args* job = start<true>(jobs, c);
    if (!job) return;
    const Args& args = *job;
    const LinPass& p = args.p;
    if (c.sg.j + 1 >= c.sg.count || c.sg.u + c.sg.j >= lin::seg_rows(p.total_T, p.seg_len)) return;
    auto load = [&](int i) {
        uint8_t* st = c.sm + i % STATE_STAGES * 2 * TILE;
        uint64_t* full = &c.b->full[i % STATE_STAGES];
        const int tok = (int)chunk_start(c, i);
        mbar_arrive_expect_tx(full, 2 * TILE);
        load_tile(&args.y, st, c.h, tok, full);
        load_tile(&args.z, st + TILE, c.h, tok, full);
    };
    set_up(args, c, 16, 16, [&] {
        for (int i = 0; i < c.chunks && i < STATE_STAGES; ++i) load(i);
    });
    Bars* b = c.b;
    const int tid = threadIdx.x, warp = tid >> 5, n = c.chunks;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    if (warp == 16) {
        if ((tid & 31) == 0) {
            int issued = n < STATE_STAGES ? n : STATE_STAGES;
            for (int i = issued; i < n; ++i) {
                if (!wait1(b, &b->empty[i % STATE_STAGES], (i / STATE_STAGES - 1) & 1, p, 331))
                    break;
                load(i);
                issued = i + 1;
            }
            for (int i = issued > STATE_STAGES ? issued - STATE_STAGES : 0; i < issued; ++i)
                mbar_wait(&b->full[i % STATE_STAGES], (i / STATE_STAGES) & 1, nullptr);
            if (!b->abort && wait1(b, &b->end, 0, p, 337)) {
                store_states(&args.segs, c.sm, (int)((c.sg.u + c.sg.j) * p.H + c.h));
                bulk_wait<false>();
            }
        }
    } else if (warp == 17) {
        constexpr uint32_t id = idesc_bf16(D, D, 0, 1);
        for (int i = 0; i < n; ++i) {
            const int s = i % STATE_STAGES;
            const uint32_t z = tile_mn(smem_u32(c.sm) + s * 2 * TILE + TILE);
            const uint32_t w = TS_W + 192 * (i & 1);
            if (!wait_warp(b, &b->full[s], (i / STATE_STAGES) & 1, p, 332)) break;
            if (!wait_warp(b, &b->w[i & 1], (i >> 1) & 1, p, 333)) break;
            const bool fresh = i % JOIN == 0;
            if (fresh && i > 0 && !wait_warp(b, &b->joined, (i / JOIN - 1) & 1, p, 338)) break;
            fence_proxy_async();   // rows of z that were zeroed
            tc_fence_after();
            if (fresh) {
                product_ta<false>(TS_U, w + 128, z, id);
            } else {
                product_ta<true>(TS_U, w + 128, z, id);
            }
            product_ta<true>(TS_U, w + 64, z, id);
            product_ta<true>(TS_U, w, z, id);
#pragma unroll
            for (int kk = 1; kk < 8; ++kk)
#pragma unroll
                for (int part = 2; part >= 0; --part)
                    product_ta<true>(TS_U, w + 64 * part + 8 * kk, z + step_mn(kk),
                                     id);
            commit(&b->wfree[i & 1]);
            commit(&b->empty[s]);
        }
        commit(&b->fin);
        mbar_wait(&b->fin, 0, nullptr);
    } else {
        const int r = tid & 127, grp = tid >> 7;
        bool ok = true;
        float sum[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[j] = 0.0f;
        auto join = [&] {      // what TMEM holds joins the sums
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t v[16];
                tmem_ld16(lanes + TS_U + 32 * grp + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[16 * q + j] += __uint_as_float(v[j]);
            }
            tc_fence_before();
        };
        for (int i = 0; i < n; ++i) {
            const int s = i % STATE_STAGES, buf = i & 1;
            const int64_t tok = chunk_start(c, i);
            const int len = chunk_len(c, tok);
            const float f = lin::decay_pow(c.g, c.rev ? tok - c.sg.t0 : c.sg.t1 - (tok + len));
            if (!(ok = wait_warp(b, &b->full[s], (i / STATE_STAGES) & 1, p, 334))) break;
            if (i >= 2 && !(ok = wait_warp(b, &b->wfree[buf], ((i >> 1) - 1) & 1, p, 335))) break;
            tc_fence_after();
            uint8_t* y = c.sm + s * 2 * TILE;
            if (len < C) zero_rows(y + TILE, len, tid, 512);
            const float* wt = c.wtab + (c.rev ? 0 : C - len);
            const uint32_t w = lanes + TS_W + 192 * buf + 16 * grp;
            split_w(smem_u32(y), warp & 3, 32 * grp, wt, f, len, w, w + 64, w + 128);
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&b->w[buf]);
            if (i > 0 && i % JOIN == 0) {
                // (the next chunk's buffer would wait for the same products)
                if (!(ok = wait_warp(b, &b->wfree[buf ^ 1], ((i - 1) >> 1) & 1, p, 339))) break;
                join();
                arrive_warp(&b->joined);
            }
        }
        if (ok && wait_warp(b, &b->fin, 0, p, 336)) {
            join();
#pragma unroll
            for (int j = 0; j < 32; j += 4)   // (the stages are read)
                store_state(c.sm, r, 32 * grp + j, sum + j);
            arrive_warp(&b->end);
        }
    }
    finish(c, 16);
}

// A tensor [n2][n1][128] cut into boxes of b2 x b1 rows of 128 bytes, swizzled as the
// tensor core's operands are.
bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t n1, int64_t n2,
              uint32_t b1, uint32_t b2) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                         cudaEnableDefault, &found) == cudaSuccess &&
                        found == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    if (!encode || n1 > INT_MAX || n2 > INT_MAX) return false;
    const cuuint64_t eb = type == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 ? 2 : 4;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {D * eb, D * eb * (cuuint64_t)n1};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / eb), b1, b2}, one[3] = {1, 1, 1};
    return encode(map, type, 3, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [total_T][H][128] bf16 in boxes of 128 tokens by 64 channels of one head.
bool make_row_map(CUtensorMap* map, const void* base, const LinPass& p) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, p.H, p.total_T, 1, C);
}
// `count` fp32 states [128][128] in boxes of all rows by 32 columns.
bool make_state_map(CUtensorMap* map, const float* base, int64_t count) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base, D, count, D, 1);
}

bool make_args(Args* a, const LinPass& p) {
    a->p = p;
    return make_row_map(&a->x, p.x, p) &&
           make_row_map(&a->y, p.y, p) &&
           make_row_map(&a->z, p.z, p) &&
           make_row_map(&a->out, p.out, p) &&
           (!p.state_in || make_state_map(&a->init, p.state_in, (int64_t)p.N * p.H)) &&
           (!p.state_out || make_state_map(&a->last, p.state_out, (int64_t)p.N * p.H)) &&
           (p.total_T < p.seg_len ||
            make_state_map(&a->segs, p.seg_states, (int64_t)(p.total_T / p.seg_len) * p.H));
}

}  // namespace

cudaError_t launch_lin_pass_tc(const LinPass* passes, int n, cudaStream_t stream) {
    Jobs jobs;
    memset(&jobs, 0, sizeof(jobs));
    jobs.n = n;
    jobs.first = 1;
    for (int i = 0; i < n; ++i) {
        if (!make_args(&jobs.a[i], passes[i])) return cudaErrorInvalidValue;
    }
    const LinPass& p = passes[0];
    const int64_t most = (int64_t)p.total_T / p.seg_len;   // segments that are not a last one
    const int64_t units = (int64_t)p.H * n;
    const int64_t grid = (p.lead > 0 ? 2 * (int64_t)p.N : most + p.N) * units;
    const int64_t state_grid = p.lead > 0 ? (int64_t)p.N * p.lead * units : grid;
    if (grid > INT_MAX || state_grid > INT_MAX) return cudaErrorInvalidConfiguration;
    cudaError_t err;
    if (most > 0) {
        err = cudaFuncSetAttribute(lin_states_tc_kernel,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (err != cudaSuccess) return err;
        lin_states_tc_kernel<<<(unsigned)state_grid, STATE_THREADS, SMEM, stream>>>(jobs);
        jobs.first = 0;
        err = launch_lin_scan(passes, n, stream);
        if (err != cudaSuccess) return err;
    }
    err = cudaFuncSetAttribute(lin_pass_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               SMEM);
    if (err != cudaSuccess) return err;
    if (most > 0) return launch_follower(lin_pass_tc_kernel, (unsigned)grid, THREADS, SMEM, stream, jobs);
    lin_pass_tc_kernel<<<(unsigned)grid, THREADS, SMEM, stream>>>(jobs);
    return cudaGetLastError();
}

}  // namespace kda
