// kda_lin.h -- declarations of the decayed linear attention, shared by its
// C-ABI layer (kda_lin_api.cpp) and its kernels.  Not part of the public
// interface.
//
// Forward and backward are one kind of pass.  With a = e^{g_h},
//     out_t = out_scale * ( sum_{s <= t} kv_scale a^{t-s} (x_t . y_s) z_s
//                           + a^{(tokens before t) + 1} S_in^T x_t )
// over rows x, y of width dx and z, out of width dz:
//   o  : x, y, z = q, k, v      S_in = S_0
//   dq : x, y, z = dO, v, k     S_in = S_0^T
//   dk : x, y, z = v, dO, q     S_in = dS_T^T, time reversed
//   dv : x, y, z = k, q, dO     S_in = dS_T,   time reversed; S_out = dS_0
// In a reversed pass t and s run from each sequence's end and the carried
// state is already decayed when it is handed on: the token that meets S_in
// first weights it with a^0, and S_out ends with one factor a more.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

struct LinPass {
    const void* x;              // [total_T, H, dx]
    const void* y;              // [total_T, H, dx]
    const void* z;              // [total_T, H, dz]
    void* out;                  // [total_T, H, dz]
    const float* log_decay;     // [H]
    const float* state_in;      // [N, H, dx, dz] (or [N, H, dz, dx]), or null
    float* state_out;           // [N, H, dx, dz], or null
    float* seg_states;          // workspace [total_T / seg_len][H][dx][dz]
    const int32_t* cu_seqlens;  // device [N + 1], or null (equal lengths)
    int32_t* status;            // workspace status word
    int32_t N;
    int32_t total_T;
    int32_t H;
    int32_t dx;
    int32_t dz;
    int32_t seg_len;            // tokens per segment, a multiple of 128
    int32_t lead;               // segments of a sequence's head where it is cut in two, else 0
    int32_t state_in_turned;    // state_in holds [dz, dx]
    int32_t reverse;
    float out_scale;
    float kv_scale;
};

// The cut of the sequences for these sizes: every one is cut into segments of
// seg_len tokens so that a few long sequences still fill `sms` SMs.
// `ctas_per_pair`: CTAs that work on one (sequence, head) pair without a cut;
// `ctas_per_sm`: how many an SM is to get.
struct LinCut {
    int32_t seg_len;
    int32_t lead;
};
LinCut lin_cut(int32_t N, int32_t total_T, int32_t H, int ctas_per_pair, int ctas_per_sm, int sms);
// The cut for the pass on the tensor cores (one CTA an SM).  Where the pairs fill
// more than half of the SMs but not all, each sequence is cut in two: a head of
// `lead` segments, and a tail.  The idle SMs work on heads, k of them one after
// another while a tail, k times as long, runs; the states before the tails come
// first, from the heads' segments over all SMs.
LinCut lin_cut_tc(int32_t N, int32_t total_T, int32_t H, int passes, int sms);

// Up to three passes on the CUDA cores, fp32 arithmetic: dx, dz in {32, 64, 128},
// dtype 0 = fp32, 1 = bf16.  Same sequences, heads and dx dz; sizes of segments and
// their states each their own.
cudaError_t launch_lin_pass(const LinPass* passes, int n, int dtype, cudaStream_t stream);
// The pass on the tensor cores: bf16, dx = dz = 128, total_T > 0.  A wait that
// ran out leaves a nonzero status word.
// Up to three passes of the same sizes and sequences run as one.
cudaError_t launch_lin_pass_tc(const LinPass* passes, int n, cudaStream_t stream);

// Turns the states that the segments add into the states before the segments:
// row u + j of seg_states, the sum of segment j alone, becomes the state before
// segment j + 1 (in pass order).
cudaError_t launch_lin_scan(const LinPass* passes, int n, cudaStream_t stream);

// One decode token per row, the state pool updated in place.
struct LinDecode {
    const void* q;              // [B, H, d_k]
    const void* k;
    const void* v;              // [B, H, d_v]
    const float* log_decay;     // [H]
    float* state;               // [pool_size, H, d_k, d_v]
    const int32_t* slots;       // [B] or null
    void* o;                    // [B, H, d_v]
    int32_t pool_size;
    int32_t B;
    int32_t H;
    float scale;
};
cudaError_t launch_lin_decode(const LinDecode& p, int d_k, int d_v, int dtype,
                              cudaStream_t stream);

}  // namespace kda
