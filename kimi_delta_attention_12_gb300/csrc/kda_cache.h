// kda_cache.h -- declarations of the rotary positions and of the paged 8-bit cache, shared
// by their C-ABI layer (kda_cache_api.cpp) and their kernels.  Not part of the public
// interface.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct Rotary {
    const void* x[2];          // q, k (or null)
    void* out[2];
    int64_t stride[2];         // between rows, in elements
    int64_t out_stride[2];
    int32_t heads[2];
    const int32_t* positions;  // [T]
    const float* inv_freq;     // [rot / 2]
    int64_t T;
    int32_t d, rot, first;
    int32_t interleaved, inverse;
    float magnitude;
};

cudaError_t launch_rotary(const Rotary& p, int dtype, cudaStream_t stream);

struct CachePlan {
    const int32_t* past;
    const int32_t* fresh;      // new tokens, -1: the request ends
    int32_t N;
    int32_t* table;
    int32_t width;
    int32_t* free_blocks;
    int32_t capacity;
    const int32_t* n_free;
    int32_t* n_free_out;
    int32_t block_log2;
    int32_t T;
    int32_t* cu;
    int32_t* context;
    int32_t* positions;
    int32_t* slots;
    int32_t* status;
};

cudaError_t launch_cache_plan(const CachePlan& p, cudaStream_t stream);

struct CacheWrite {
    const void* x[2];          // k, v
    int64_t stride[2];
    uint8_t* cache[2];
    float* scale[2];
    const int32_t* slots;
    int32_t T, heads, d;
    int32_t num_blocks, block_log2;
};

cudaError_t launch_cache_write(const CacheWrite& p, int dtype, cudaStream_t stream);

struct CacheAttention {
    const void* q;
    int64_t q_stride;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const float* k_scale;
    const float* v_scale;
    int32_t num_blocks, block_log2;
    const int32_t* table;
    int32_t width;
    const int32_t* context;
    const int32_t* cu;         // or null: one new token each
    int32_t N, T, max_new;
    int32_t heads, group;      // key and value heads; query heads to each
    int32_t d;
    float scale;
    void* o;
    // workspace: a status word, which the call's first kernel clears, and partial sums
    int32_t* status;
    int32_t clears;
    float* partial;
    float* prompt_partial;     // of the prompts' kernel
    int64_t many_rows;         // rows (heads of a group times new tokens) of a request from which
                               // on the prompts' kernel takes it, the other one below
};

// Whether the prompts' kernel has a form for these.
bool cache_prompt_takes(int32_t d, int dtype);
size_t cache_prompt_room(int32_t d, int sms);
// The kernel, and what joins its parts: launched behind it, or behind one that waits for it.
cudaError_t launch_cache_prompt(const CacheAttention& p, int sms, cudaStream_t stream);
cudaError_t launch_cache_prompt_join(const CacheAttention& p, int sms, cudaStream_t stream);
// Whether a call's prompts may go to it: so many rows in all, and in the longest request.
bool cache_prompt_used(int32_t heads, int32_t group, int32_t T, int32_t max_new, int32_t d,
                       int dtype);
// Bytes of partial sums, on a device of that many SMs.
size_t cache_attention_room(int32_t heads, int32_t group, int32_t T, int32_t max_new, int32_t d,
                            int dtype, int sms);
cudaError_t launch_cache_attention(const CacheAttention& p, int dtype, int sms,
                                   cudaStream_t stream);

}  // namespace kda
