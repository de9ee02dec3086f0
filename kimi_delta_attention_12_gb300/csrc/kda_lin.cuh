// kda_lin.cuh -- device helpers of the decayed linear attention: powers of
// the decay and the cut of packed sequences into segments.
#pragma once

#include <stdint.h>

#include "kda_seqlens.cuh"

namespace kda {
namespace lin {

// e^{g n}, n >= 0.  The product's rounding error is carried into the factor
// (e^{p + err} = e^p (1 + err)), so a long distance costs no digits; n = 0 is
// 1 whatever g is (an infinite g means a state that is dropped every token).
__device__ __forceinline__ float decay_pow(float g, int64_t n) {
    if (n == 0) return 1.0f;
    const float fn = (float)n, p = g * fn;
    if (p < -200.0f) return 0.0f;
    const float err = fmaf(g, fn, -p);
    return fabsf(err) < 1.0f ? expf(p) * (1.0f + err) : expf(p);
}

// A segment of a sequence in the order of the pass.
struct Segment {
    int n;            // sequence, or -1: no such segment
    int j;            // position among the sequence's segments, in pass order
    int count;        // the sequence's segments
    int64_t bos, eos; // its sequence's tokens
    int64_t t0, t1;   // its own tokens
    int64_t u;        // row of seg_states of the sequence's segment 0
};

__device__ __forceinline__ int seg_count(int64_t len, int64_t seg_len) {
    return len <= seg_len ? 1 : (int)((len + seg_len - 1) / seg_len);
}

// Token range of the sequence's segment i in pass order.
__device__ __forceinline__ void seg_tokens(const Segment& s, int i, int64_t seg_len, int reverse,
                                           int64_t& t0, int64_t& t1) {
    const int k = reverse ? s.count - 1 - i : i;
    t0 = s.bos + (int64_t)k * seg_len;
    t1 = t0 + seg_len < s.eos ? t0 + seg_len : s.eos;
}

// Rows of seg_states: each sequence keeps the states of all its segments but
// the last one, at most floor(length / seg_len) of them.
__device__ __forceinline__ int64_t seg_rows(int64_t total_T, int64_t seg_len) {
    return total_T / seg_len;
}

// Segment number `index` over all sequences (sequence by sequence; an empty
// sequence has one empty segment).  Every warp calls it whole.
__device__ __forceinline__ Segment find_segment(const int32_t* cu, int N, int64_t total_T,
                                                int64_t seg_len, int reverse, int64_t index) {
    Segment s;
    s.n = -1;
    s.j = s.count = 0;
    s.bos = s.eos = s.t0 = s.t1 = s.u = 0;
    if (!cu) {
        const int64_t len = total_T / N;
        s.count = seg_count(len, seg_len);
        if (index >= (int64_t)N * s.count) return s;
        s.n = (int)(index / s.count);
        s.j = (int)(index % s.count);
        s.u = (int64_t)s.n * (s.count - 1);
        s.bos = s.n * len;
        s.eos = s.bos + len;
    } else {
        const int lane = threadIdx.x & 31;
        int64_t before = 0;   // segments of the sequences before this round's
        for (int base = 0; base < N; base += 32) {
            const int n = base + lane;
            const int c = n < N ? seg_count(clamped_len(cu, n, N, total_T), seg_len) : 0;
            int sum = c;
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += o;
            }
            const int64_t first = before + sum - c;
            const unsigned hit = __ballot_sync(0xffffffffu, index >= first && index < first + c);
            if (hit) {
                const int src = __ffs(hit) - 1;
                const int64_t f = before + __shfl_sync(0xffffffffu, sum - c, src);
                s.n = base + src;
                s.j = (int)(index - f);
                s.count = __shfl_sync(0xffffffffu, c, src);
                s.u = f - s.n;   // every sequence before it keeps all segments but one
                clamped_seq(cu, s.n, N, total_T, s.bos, s.eos);
                break;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (s.n < 0) return s;
    }
    seg_tokens(s, s.j, seg_len, reverse, s.t0, s.t1);
    return s;
}

// The sequence of rank k by length, longest first (equal ones in order), of up to
// RANKED sequences; N past them.  Every warp calls it whole.
constexpr int RANKED = 64;
__device__ __forceinline__ int nth_longest(const int32_t* cu, int N, int64_t total_T, int k) {
    if (k >= N) return N;
    const int lane = threadIdx.x & 31;
    const int64_t a = lane < N ? clamped_len(cu, lane, N, total_T) : -1;
    const int64_t b = lane + 32 < N ? clamped_len(cu, lane + 32, N, total_T) : -1;
    int ra = 0, rb = 0;
    for (int j = 0; j < N; ++j) {
        const int64_t l = __shfl_sync(0xffffffffu, j < 32 ? a : b, j & 31);
        ra += l > a || (l == a && j < lane);
        rb += l > b || (l == b && j < lane + 32);
    }
    const unsigned ha = __ballot_sync(0xffffffffu, lane < N && ra == k);
    const unsigned hb = __ballot_sync(0xffffffffu, lane + 32 < N && rb == k);
    return ha ? __ffs(ha) - 1 : 31 + __ffs(hb);
}

// The first segment of sequence n.  Every warp calls it whole.
__device__ __forceinline__ Segment first_segment(const int32_t* cu, int N, int64_t total_T,
                                                 int64_t seg_len, int reverse, int n) {
    Segment s;
    s.n = n;
    s.j = 0;
    s.u = 0;
    clamped_seq(cu, n, N, total_T, s.bos, s.eos);
    s.count = seg_count(s.eos - s.bos, seg_len);
    if (!cu) {
        s.u = (int64_t)n * (s.count - 1);
    } else {
        int64_t u = 0;
        for (int m = threadIdx.x & 31; m < n; m += 32)
            u += seg_count(clamped_len(cu, m, N, total_T), seg_len) - 1;
        for (int d = 16; d > 0; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
        s.u = u;
    }
    seg_tokens(s, 0, seg_len, reverse, s.t0, s.t1);
    return s;
}

// Sequence n cut in two, a head of `lead` segments and a tail (n < 0: no such
// part).  The state before the tail is the one after segment lead - 1; a
// sequence of no more than `lead` segments is all head.
__device__ __forceinline__ Segment half_segment(const int32_t* cu, int N, int64_t total_T,
                                                int64_t seg_len, int reverse, int lead, int n,
                                                bool tail) {
    Segment s = first_segment(cu, N, total_T, seg_len, reverse, n);
    const bool two = s.count > lead;
    if (tail && !two) s.n = -1;
    const int64_t at = reverse ? s.bos + (s.count - lead) * seg_len : s.bos + lead * seg_len;
    s.t0 = s.bos;
    s.t1 = s.eos;
    if (two) (tail != (reverse != 0) ? s.t0 : s.t1) = at;
    s.j = tail ? lead : 0;
    s.count = two ? lead + 1 : 1;
    return s;
}

// Segment j of the head of sequence n, where there is a tail behind it.
__device__ __forceinline__ Segment lead_segment(const int32_t* cu, int N, int64_t total_T,
                                                int64_t seg_len, int reverse, int lead, int n,
                                                int j) {
    Segment s = first_segment(cu, N, total_T, seg_len, reverse, n);
    if (s.count <= lead) s.n = -1;
    s.j = j;
    seg_tokens(s, j, seg_len, reverse, s.t0, s.t1);
    return s;
}

}  // namespace lin
}  // namespace kda
