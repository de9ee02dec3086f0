// kda_block_norm.h -- declarations of the block norms, shared by their C-ABI
// layer (kda_norm_api.cpp) and their kernels.  Not part of the public
// interface.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct BlockNorm {
    const void* y;            // [rows, D]
    const float* w_post;      // [group]
    const void* gate;         // [rows, D] or null
    const void* x;            // forward: the stream before; backward: x_out as stored; or null
    const float* res_scale;   // [D] or null (1)
    const float* w_pre;       // [D] or null (no h)
    int64_t rows;
    int32_t D;
    int32_t group;            // channels per norm of y: D, or 32, 64, 128
    int32_t silu;             // gate: silu instead of sigmoid
    float eps;
    // forward
    void* x_out;              // [rows, D]
    void* h;                  // [rows, D] with w_pre
    // backward
    const void* dx_out;       // [rows, D] or null (zero)
    const void* dh;           // [rows, D] with w_pre
    void* dy;                 // [rows, D]
    void* dgate;              // [rows, D] with a gate
    void* dx;                 // [rows, D] or null
    float* dw_post;           // [group]
    float* dres_scale;        // [D] with res_scale
    float* dw_pre;            // [D] with w_pre
    float* partial;           // workspace [block_norm_parts][3][D]
};

// Row groups whose sums of the weights' gradients are kept apart (a bound on
// the backward's grid, the same on every device).
int block_norm_parts(int64_t rows, int32_t D);
cudaError_t launch_block_norm(const BlockNorm& p, int dtype, cudaStream_t stream);
cudaError_t launch_block_norm_backward(const BlockNorm& p, int dtype, cudaStream_t stream);

}  // namespace kda
