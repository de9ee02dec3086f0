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
// Roles: warps 0-3 turn P into P' and write the outputs (thread = token);
// warps 4-7 split w Y and carry the state (thread = row of S); warp 8 issues
// the TMA loads, warp 9 the products.
#include "kda_lin.h"

#include <cuda.h>
#include <cuda_bf16.h>
#include <limits.h>
#include <string.h>

#include "kda_chunked.h"
#include "kda_lin.cuh"
#include "sm103_ptx.cuh"

namespace kda {
namespace {

using namespace sm103;

constexpr int C = 128;                   // tokens per chunk = rows of a tile
constexpr int D = 128;                   // dx = dz
constexpr int THREADS = 320;
constexpr uint32_t HALF = C * 128;       // a tile's 64 columns: 128 rows of 128 bytes
constexpr uint32_t TILE = 2 * HALF;
constexpr int STAGES = 2;                // the pass: X, Y, Z per stage
constexpr int STATE_STAGES = 3;          // the segment states: Y, Z per stage
constexpr uint32_t SM_S = STAGES * 3 * TILE;             // bf16 copy of the state
constexpr uint32_t SM_TAB = SM_S + TILE;
static_assert(SM_S >= STATE_STAGES * 2 * TILE, "the states' stages end before the copy");
constexpr uint32_t SMEM = SM_TAB + 2048 + 1024;          // tables, alignment
static_assert(SMEM <= 232448, "more shared memory than a CTA may have");

// TMEM columns of the pass
constexpr uint32_t TC_P = 0;             // P; P' (bf16 pairs) in its first 64 columns
constexpr uint32_t TC_O = 128;           // P' Z
constexpr uint32_t TC_U = 256;           // X S, then (w Y)^T Z
constexpr uint32_t TC_W = 384;           // w Y: tokens 0-63 in three parts of 32 columns,
                                         // tokens 64-127: first part, the others ...
constexpr uint32_t TC_W2 = 64;           // ... where P was
// and of the segment states
constexpr uint32_t TS_U = 0;
constexpr uint32_t TS_W = 128;           // two buffers of three parts of 64 columns

static_assert((132 + 132) * 4 + 256 <= 2048, "tables and barriers");

struct Args {
    CUtensorMap x, y, z;
    LinPass p;
};

struct Bars {
    uint64_t full[STATE_STAGES];   // tiles of a stage are there
    uint64_t empty[STATE_STAGES];  // products on a stage are done
    uint64_t qk, o1, o2, u;        // P / X S / P' Z / (w Y)^T Z done
    uint64_t p, s, o1r, wa, wb;    // P' / S copy / X S read / w Y first and second half written
    uint64_t w[2], wfree[2];       // segment states: w Y of a buffer written, read
    uint64_t fin;
    uint32_t tmem;
    volatile int abort;
};

static_assert(sizeof(Bars) <= 256, "barriers");

__device__ __forceinline__ void give_up(const LinPass& p, Bars* b, int site) {
    atomicCAS(p.status, 0, site);
    b->abort = 1;
}

// One thread's bounded wait; on a timeout every role of the CTA leaves its loop.
__device__ __forceinline__ bool wait1(Bars* b, uint64_t* bar, uint32_t parity, const LinPass& p,
                                      int site) {
    if (mbar_wait(bar, parity, &b->abort)) return true;
    give_up(p, b, site);
    return false;
}

// The same for a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool wait_warp(Bars* b, uint64_t* bar, uint32_t parity,
                                          const LinPass& p, int site) {
    const bool ok = mbar_wait(bar, parity, &b->abort);
    if (__all_sync(0xffffffffu, ok)) return true;
    give_up(p, b, site);
    return false;
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// K-major operand: rows of 64 channels; k-step kk covers 16 channels.
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int kk) {
    return smem_desc(tile + (kk >> 2) * HALF + (kk & 3) * 32, 16, 1024);
}
// MN-major operand: rows are the summed index; k-step kk covers 16 rows.
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int kk) {
    return smem_desc(tile + kk * 2048, HALF, 1024);
}

// w Y of one row of S for 64 tokens, split into three bf16 parts: column pairs
// of tokens to TMEM.  w: the weight of token 0, those of the others up (REV) or
// down from there.  Rows past the chunk's end (another sequence's, maybe not
// finite) count as zero; their weights are read from the table below.
template <bool REV>
__device__ __forceinline__ void split_w(const uint8_t* y, int r, int tok0, const float* w, float f,
                                        int len, uint32_t hi, uint32_t mid, uint32_t lo) {
    const uint8_t* col = y + (r >> 6) * HALF;
    const uint32_t at = (r & 63) * 2;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        uint32_t h[8], m[8], l[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int s = tok0 + 16 * b + 2 * j;
            const float w0 = w[REV ? s : -s], w1 = w[REV ? s + 1 : -s - 1];
            const uint32_t k0 = *reinterpret_cast<const uint16_t*>(col + sw128(s, at));
            const uint32_t k1 = *reinterpret_cast<const uint16_t*>(col + sw128(s + 1, at));
            float x0 = __uint_as_float(k0 << 16) * (w0 * f);
            float x1 = __uint_as_float(k1 << 16) * (w1 * f);
            if (s >= len) x0 = 0.0f;
            if (s + 1 >= len) x1 = 0.0f;
            h[j] = pack(x0, x1);
            x0 -= low(h[j]);
            x1 -= high(h[j]);
            m[j] = pack(x0, x1);
            l[j] = pack(x0 - low(m[j]), x1 - high(m[j]));
        }
        tmem_st8(hi + 8 * b, h);
        tmem_st8(mid + 8 * b, m);
        tmem_st8(lo + 8 * b, l);
    }
}

// Rows len .. 127 of a Z tile to zero: they meet zeros of P' and w Y, and may
// hold another sequence's values, which need not be finite.
__device__ __forceinline__ void zero_rows(uint8_t* z, int len, int tid) {
    for (int i = tid; i < (C - len) * 16; i += 128) {
        const int row = len + (i >> 4), part = i & 15;
        *reinterpret_cast<uint4*>(z + (part >> 3) * HALF + row * 128 + (part & 7) * 16) =
            make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
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
    float* lam;     // a^0 .. a^128
    float* lamk;    // the same times kv_scale (behind lam: see split_w)
    lin::Segment sg;
    int h, chunks;
    float g;
};

__device__ __forceinline__ bool start(const Args& args, Cta& c) {
    extern __shared__ uint8_t smem_raw[];
    const LinPass& p = args.p;
    c.sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~(uintptr_t)1023);
    c.lam = reinterpret_cast<float*>(c.sm + SM_TAB);
    c.lamk = c.lam + 132;
    c.b = reinterpret_cast<Bars*>(c.lamk + 132);
    c.h = blockIdx.x % p.H;
    c.sg = lin::find_segment(p.cu_seqlens, p.N, p.total_T, p.seg_len, p.reverse,
                             blockIdx.x / p.H);
    return c.sg.n >= 0;
}

__device__ __forceinline__ void set_up(const Args& args, Cta& c) {
    const LinPass& p = args.p;
    const int tid = threadIdx.x;
    c.chunks = (int)((c.sg.t1 - c.sg.t0 + C - 1) / C);
    c.g = p.log_decay[c.h];
    if (tid <= C) {
        const float a = lin::decay_pow(c.g, tid);
        c.lam[tid] = a;
        c.lamk[tid] = a * p.kv_scale;
    }
    if (tid == 288) {
        Bars* b = c.b;
        for (int i = 0; i < STATE_STAGES; ++i) {
            mbar_init(&b->full[i], 1);
            mbar_init(&b->empty[i], 1);
        }
        uint64_t* one[] = {&b->qk, &b->o1, &b->o2, &b->u, &b->wfree[0], &b->wfree[1], &b->fin};
        uint64_t* all[] = {&b->p, &b->s, &b->o1r, &b->wa, &b->wb, &b->w[0], &b->w[1]};
        for (uint64_t* x : one) mbar_init(x, 1);
        for (uint64_t* x : all) mbar_init(x, 128);
        b->abort = 0;
        fence_mbar_init();
    }
    if (tid >> 5 == 8) {
        tmem_alloc(&c.b->tmem, 512);
        tmem_relinquish();
        if ((tid & 31) == 0) {
            prefetch_tmap(&args.x);
            prefetch_tmap(&args.y);
            prefetch_tmap(&args.z);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

__device__ __forceinline__ void finish(const Cta& c, uint32_t tmem) {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x >> 5 == 8) tmem_dealloc(tmem, 512);
}

// Token range of the pass's step i.
__device__ __forceinline__ int64_t chunk_start(const Cta& c, int reverse, int i) {
    return c.sg.t0 + (int64_t)(reverse ? c.chunks - 1 - i : i) * C;
}
__device__ __forceinline__ int chunk_len(const Cta& c, int64_t tok) {
    return (int)(c.sg.t1 - tok < C ? c.sg.t1 - tok : C);
}

// ------------------------------------------------------------------ the pass
template <bool REV>
__global__ void __launch_bounds__(THREADS, 1) lin_pass_tc_kernel(const __grid_constant__ Args args) {
    const LinPass& p = args.p;
    Cta c;
    if (!start(args, c)) return;
    set_up(args, c);
    Bars* b = c.b;
    const uint32_t tmem = b->tmem;
    const int tid = threadIdx.x, warp = tid >> 5, n = c.chunks;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);   // this warp's 32 TMEM lanes

    if (warp == 8) {
        if ((tid & 31) == 0) {
            int issued = 0;
            for (int i = 0; i < n; ++i) {
                const int s = i & 1;
                if (i >= STAGES && !wait1(b, &b->empty[s], ((i >> 1) - 1) & 1, p, 301)) break;
                uint8_t* st = c.sm + s * 3 * TILE;
                const int tok = (int)chunk_start(c, REV, i);
                mbar_arrive_expect_tx(&b->full[s], 3 * TILE);
                load_tile(&args.x, st, c.h, tok, &b->full[s]);
                load_tile(&args.y, st + TILE, c.h, tok, &b->full[s]);
                load_tile(&args.z, st + 2 * TILE, c.h, tok, &b->full[s]);
                issued = i + 1;
            }
            for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
                mbar_wait(&b->full[i & 1], (i >> 1) & 1, nullptr);   // no copy outlives the CTA
        }
    } else if (warp == 9) {
        if ((tid & 31) == 0) {
            const uint32_t id_kk = idesc_bf16(D, D, 0, 0), id_km = idesc_bf16(D, D, 0, 1);
            const uint32_t base = smem_u32(c.sm), sb = base + SM_S;
            for (int i = 0; i < n; ++i) {
                const uint32_t ph = i & 1, x = base + (i & 1) * 3 * TILE, y = x + TILE,
                               z = y + TILE;
                if (!wait1(b, &b->full[i & 1], (i >> 1) & 1, p, 302)) break;
                if (i > 0 && !wait1(b, &b->u, (i - 1) & 1, p, 303)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16(tmem + TC_P, desc_k(x, kk), desc_k(y, kk), id_kk, kk > 0);
                mma_commit(&b->qk);
                if (!wait1(b, &b->s, ph, p, 304)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16(tmem + TC_U, desc_k(x, kk), desc_mn(sb, kk), id_km, kk > 0);
                mma_commit(&b->o1);
                if (!wait1(b, &b->p, ph, p, 305)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16_ta(tmem + TC_O, tmem + TC_P + 8 * kk, desc_mn(z, kk), id_km, kk > 0);
                mma_commit(&b->o2);
                if (!wait1(b, &b->o1r, ph, p, 306)) break;
                if (!wait1(b, &b->wa, ph, p, 307)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int part = 2; part >= 0; --part)
                        mma_bf16_ta(tmem + TC_U, tmem + TC_W + 32 * part + 8 * kk, desc_mn(z, kk),
                                    id_km, kk > 0 || part < 2);
                if (!wait1(b, &b->wb, ph, p, 308)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16_ta(tmem + TC_U, tmem + TC_W2 + 32 + 8 * kk, desc_mn(z, kk + 4), id_km,
                                1);
                    mma_bf16_ta(tmem + TC_U, tmem + TC_W2 + 8 * kk, desc_mn(z, kk + 4), id_km, 1);
                    mma_bf16_ta(tmem + TC_U, tmem + TC_W + 96 + 8 * kk, desc_mn(z, kk + 4), id_km,
                                1);
                }
                mma_commit(&b->u);
                mma_commit(&b->empty[i & 1]);
            }
            mma_commit(&b->fin);
            mbar_wait(&b->fin, 0, nullptr);   // no product outlives the CTA
        }
    } else if (warp < 4) {
        const int t = tid;
        for (int i = 0; i < n; ++i) {
            const uint32_t ph = i & 1;
            const int64_t tok = chunk_start(c, REV, i);
            const int len = chunk_len(c, tok);
            if (len < C) {
                if (!wait_warp(b, &b->full[i & 1], (i >> 1) & 1, p, 310)) break;
                zero_rows(c.sm + (i & 1) * 3 * TILE + 2 * TILE, len, tid);
            }
            if (!wait_warp(b, &b->qk, ph, p, 311)) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 4; ++q) {     // 32 columns at a time, written where they were read
                uint32_t w[16];
                if (REV ? q >= warp : q <= warp) {
                    uint32_t r[2][16];
                    tmem_ld16(lanes + TC_P + 32 * q, r[0]);
                    tmem_ld16(lanes + TC_P + 32 * q + 16, r[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int s = 32 * q + 2 * j + e, d = REV ? s - t : t - s;
                            const float f = c.lamk[d & 127];
                            v[e] = d >= 0 && s < len
                                       ? __uint_as_float(r[j >> 3][2 * (j & 7) + e]) * f
                                       : 0.0f;
                        }
                        w[j] = pack(v[0], v[1]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = 0;
                }
                tmem_st16(lanes + TC_P + 16 * q, w);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&b->p);

            if (!wait_warp(b, &b->o1, ph, p, 312)) break;
            tc_fence_after();
            uint32_t o1[8][16];
#pragma unroll
            for (int q = 0; q < 8; ++q) tmem_ld16(lanes + TC_U + 16 * q, o1[q]);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&b->o1r);
            const float m = p.out_scale;
            const float f = t < len ? m * c.lam[REV ? len - 1 - t : t + 1] : 0.0f;
            __nv_bfloat16* out =
                static_cast<__nv_bfloat16*>(p.out) + ((size_t)(tok + t) * p.H + c.h) * D;
            if (!wait_warp(b, &b->o2, ph, p, 313)) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t r[16], w[8];
                tmem_ld16(lanes + TC_O + 16 * q, r);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = pack(f * __uint_as_float(o1[q][2 * j]) + m * __uint_as_float(r[2 * j]),
                                f * __uint_as_float(o1[q][2 * j + 1]) +
                                    m * __uint_as_float(r[2 * j + 1]));
                if (t < len) {
                    uint4* dst = reinterpret_cast<uint4*>(out + 16 * q);
                    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
            tc_fence_before();
        }
    } else {
        const int r = tid - 128;      // row of the state
        float S[D];
        const size_t state_floats = (size_t)D * D;
#pragma unroll
        for (int j = 0; j < D; ++j) S[j] = 0.0f;
        if (p.state_in) {
            const float* s0 = p.state_in + ((size_t)c.sg.n * p.H + c.h) * state_floats;
            if (p.state_in_turned) {
#pragma unroll
                for (int j = 0; j < D; ++j) S[j] = s0[(size_t)j * D + r];
            } else {
#pragma unroll
                for (int j = 0; j < D; j += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(s0 + (size_t)r * D + j);
                    S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
                }
            }
        }
        const int64_t rows = lin::seg_rows(p.total_T, p.seg_len);
        for (int k = 0; k < c.sg.j && c.sg.u + k < rows; ++k) {   // join the segments before
            int64_t a, e;
            lin::seg_tokens(c.sg, k, p.seg_len, REV, a, e);
            const float f = lin::decay_pow(c.g, e - a);
            const float* u = p.seg_states + ((c.sg.u + k) * (int64_t)p.H + c.h) * state_floats +
                             (size_t)r * D;
#pragma unroll
            for (int j = 0; j < D; j += 4) {
                const float4 v = *reinterpret_cast<const float4*>(u + j);
                S[j] = f * S[j] + v.x;
                S[j + 1] = f * S[j + 1] + v.y;
                S[j + 2] = f * S[j + 2] + v.z;
                S[j + 3] = f * S[j + 3] + v.w;
            }
        }
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const uint32_t ph = i & 1;
            const int len = chunk_len(c, chunk_start(c, REV, i));
            uint8_t* sbuf = c.sm + SM_S;
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                uint4 v;
                v.x = pack(S[8 * q], S[8 * q + 1]);
                v.y = pack(S[8 * q + 2], S[8 * q + 3]);
                v.z = pack(S[8 * q + 4], S[8 * q + 5]);
                v.w = pack(S[8 * q + 6], S[8 * q + 7]);
                *reinterpret_cast<uint4*>(sbuf + (q >> 3) * HALF + sw128(r, (q & 7) * 16)) = v;
            }
            fence_proxy_async();
            mbar_arrive(&b->s);
            if (!(ok = wait_warp(b, &b->full[i & 1], (i >> 1) & 1, p, 320))) break;
            const uint8_t* y = c.sm + (i & 1) * 3 * TILE + TILE;
            const float* w = c.lamk + (REV ? 1 : len - 1);
            split_w<REV>(y, r, 0, w, 1.0f, len, lanes + TC_W, lanes + TC_W + 32, lanes + TC_W + 64);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&b->wa);
            if (!(ok = wait_warp(b, &b->p, ph, p, 321))) break;   // P has been read
            tc_fence_after();
            split_w<REV>(y, r, 64, w, 1.0f, len, lanes + TC_W + 96, lanes + TC_W2,
                         lanes + TC_W2 + 32);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&b->wb);
            if (!(ok = wait_warp(b, &b->u, ph, p, 322))) break;
            tc_fence_after();
            const float f = c.lam[len];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t v[16];
                tmem_ld16(lanes + TC_U + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    S[16 * q + j] = f * S[16 * q + j] + __uint_as_float(v[j]);
            }
            tc_fence_before();
        }
        if (ok && p.state_out && c.sg.j + 1 == c.sg.count) {
            float* dst = p.state_out + ((size_t)c.sg.n * p.H + c.h) * state_floats + (size_t)r * D;
#pragma unroll
            for (int j = 0; j < D; j += 4)
                *reinterpret_cast<float4*>(dst + j) =
                    make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
        }
    }
    finish(c, tmem);
}

// ------------------------------------------------- the state a segment adds
// sum_j a^{tokens from j to the segment's end} kv_scale y_j z_j^T, accumulated in TMEM
// over the whole segment: the weights are taken to its end at once.  The two
// groups of four warps split w Y of every other chunk.
template <bool REV>
__global__ void __launch_bounds__(THREADS, 1)
lin_states_tc_kernel(const __grid_constant__ Args args) {
    const LinPass& p = args.p;
    Cta c;
    if (!start(args, c) || c.sg.j + 1 >= c.sg.count ||
        c.sg.u + c.sg.j >= lin::seg_rows(p.total_T, p.seg_len)) {
        return;
    }
    set_up(args, c);
    Bars* b = c.b;
    const uint32_t tmem = b->tmem;
    const int tid = threadIdx.x, warp = tid >> 5, n = c.chunks;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    if (warp == 8) {
        if ((tid & 31) == 0) {
            int issued = 0;
            for (int i = 0; i < n; ++i) {
                const int s = i % STATE_STAGES, use = i / STATE_STAGES;
                if (use > 0 && !wait1(b, &b->empty[s], (use - 1) & 1, p, 331)) break;
                uint8_t* st = c.sm + s * 2 * TILE;
                const int tok = (int)chunk_start(c, REV, i);
                mbar_arrive_expect_tx(&b->full[s], 2 * TILE);
                load_tile(&args.y, st, c.h, tok, &b->full[s]);
                load_tile(&args.z, st + TILE, c.h, tok, &b->full[s]);
                issued = i + 1;
            }
            for (int i = issued > STATE_STAGES ? issued - STATE_STAGES : 0; i < issued; ++i)
                mbar_wait(&b->full[i % STATE_STAGES], (i / STATE_STAGES) & 1, nullptr);
        }
    } else if (warp == 9) {
        if ((tid & 31) == 0) {
            const uint32_t id = idesc_bf16(D, D, 0, 1);
            for (int i = 0; i < n; ++i) {
                const int s = i % STATE_STAGES;
                const uint32_t z = smem_u32(c.sm) + s * 2 * TILE + TILE;
                const uint32_t w = tmem + TS_W + 192 * (i & 1);
                if (!wait1(b, &b->full[s], (i / STATE_STAGES) & 1, p, 332)) break;
                if (!wait1(b, &b->w[i & 1], (i >> 1) & 1, p, 333)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                    for (int part = 2; part >= 0; --part)
                        mma_bf16_ta(tmem + TS_U, w + 64 * part + 8 * kk, desc_mn(z, kk), id,
                                    i > 0 || kk > 0 || part < 2);
                mma_commit(&b->wfree[i & 1]);
                mma_commit(&b->empty[s]);
            }
            mma_commit(&b->fin);
            mbar_wait(&b->fin, 0, nullptr);
        }
    } else {
        const int r = tid & 127, grp = tid >> 7;
        const uint32_t w = lanes + TS_W + 192 * grp;
        bool ok = true;
        for (int i = grp; i < n; i += 2) {
            const int s = i % STATE_STAGES;
            const int64_t tok = chunk_start(c, REV, i);
            const int len = chunk_len(c, tok);
            const float f = lin::decay_pow(c.g, REV ? tok - c.sg.t0 : c.sg.t1 - (tok + len));
            if (!(ok = wait_warp(b, &b->full[s], (i / STATE_STAGES) & 1, p, 334))) break;
            if (i >= 2 && !(ok = wait_warp(b, &b->wfree[grp], ((i >> 1) - 1) & 1, p, 335))) break;
            tc_fence_after();
            uint8_t* y = c.sm + s * 2 * TILE;
            if (len < C) zero_rows(y + TILE, len, r);
            const float* wt = c.lamk + (REV ? 1 : len - 1);
            split_w<REV>(y, r, 0, wt, f, len, w, w + 64, w + 128);
            split_w<REV>(y, r, 64, wt, f, len, w + 32, w + 96, w + 160);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&b->w[grp]);
        }
        if (grp == 1 && ok && wait_warp(b, &b->fin, 0, p, 336)) {
            tc_fence_after();
            float* dst = p.seg_states +
                         ((c.sg.u + c.sg.j) * (int64_t)p.H + c.h) * (int64_t)(D * D) +
                         (size_t)r * D;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t v[16];
                tmem_ld16(lanes + TS_U + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<uint4*>(dst + 16 * q + j) =
                        make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            }
        }
    }
    finish(c, tmem);
}

template <bool REV>
cudaError_t launch(const Args& args, unsigned grid, bool cut, cudaStream_t stream) {
    cudaError_t err;
    if (cut) {
        err = cudaFuncSetAttribute(lin_states_tc_kernel<REV>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (err != cudaSuccess) return err;
        lin_states_tc_kernel<REV><<<grid, THREADS, SMEM, stream>>>(args);
    }
    err = cudaFuncSetAttribute(lin_pass_tc_kernel<REV>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (err != cudaSuccess) return err;
    lin_pass_tc_kernel<REV><<<grid, THREADS, SMEM, stream>>>(args);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_pass_tc(const LinPass& p, cudaStream_t stream) {
    Args args;
    memset(&args, 0, sizeof(args));
    args.p = p;
    if (!make_row_map(&args.x, p.x, p.total_T, p.H, C) ||
        !make_row_map(&args.y, p.y, p.total_T, p.H, C) ||
        !make_row_map(&args.z, p.z, p.total_T, p.H, C)) {
        return cudaErrorInvalidValue;
    }
    const int64_t most = (int64_t)p.total_T / p.seg_len;
    const int64_t grid = (most + p.N) * p.H;
    if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
    return p.reverse ? launch<true>(args, (unsigned)grid, most > 0, stream)
                     : launch<false>(args, (unsigned)grid, most > 0, stream);
}

}  // namespace kda
