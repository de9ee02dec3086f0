// kda_norm_api.cpp -- the C ABI of the block norms declared in include/kda.h:
// argument validation and launches on the caller's stream.
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "kda_block_norm.h"
#include "kda_checks.h"

namespace {

using kda::aligned;
using kda::elem_bytes;
using kda::overlaps;

constexpr int32_t kMaxNormWidth = 16384;

bool supported_norm(int32_t D, int32_t group) {
    return D >= 8 && D <= kMaxNormWidth && D % 8 == 0 &&
           (group == D || ((group == 32 || group == 64 || group == 128) && D % group == 0));
}

// What both directions check alike; KDA_OK, or the error.
int check_norm(const void* y, const float* w_post, int64_t rows, int32_t D, int32_t group,
               kda_dtype dt, int32_t gate_act, float eps) {
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (rows < 0 || D < 1 || group < 1) return KDA_ERR_INVALID_ARG;
    if (!supported_norm(D, group)) return KDA_ERR_UNSUPPORTED;
    if (gate_act != KDA_GATE_SIGMOID && gate_act != KDA_GATE_SILU) return KDA_ERR_INVALID_ARG;
    if (!isfinite(eps) || eps <= 0.0f || !w_post || (rows > 0 && !y)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_block_norm(const void* y, const float* w_post, const void* gate, const void* x,
                   const float* res_scale, const float* w_pre, int64_t rows, int32_t D,
                   int32_t group, kda_dtype dt, int32_t gate_act, float eps, void* x_out, void* h,
                   void* stream) {
    const int bad = check_norm(y, w_post, rows, D, group, dt, gate_act, eps);
    if (bad != KDA_OK) return bad;
    if ((rows > 0 && !x_out) || (rows > 0 && w_pre && !h) || (!w_pre && h)) {
        return KDA_ERR_INVALID_ARG;
    }
    const void* row[5] = {y, gate, x, x_out, h};
    const float* par[3] = {w_post, res_scale, w_pre};
    for (const void* b : row) {
        if (!aligned(b, 16)) return KDA_ERR_ALIGNMENT;
    }
    for (const float* b : par) {
        if (!aligned(b, 16)) return KDA_ERR_ALIGNMENT;
    }
    // an element is written by the thread that has read it: x_out or h may be
    // y, gate or x itself, but no other overlap is allowed
    const size_t n = (size_t)rows * D * elem_bytes(dt);
    for (int o = 3; o < 5; ++o) {
        for (int i = 0; i < o; ++i) {
            if (overlaps(row[o], n, row[i], n) && (i == 3 || row[o] != row[i])) {
                return KDA_ERR_INVALID_ARG;
            }
        }
        for (int i = 0; i < 3; ++i) {
            const size_t np = (size_t)(i == 0 ? group : D) * sizeof(float);
            if (overlaps(row[o], n, par[i], np)) return KDA_ERR_INVALID_ARG;
        }
    }
    if (rows == 0) return KDA_OK;
    kda::BlockNorm p;
    memset(&p, 0, sizeof(p));
    p.y = y; p.w_post = w_post; p.gate = gate; p.x = x; p.res_scale = res_scale; p.w_pre = w_pre;
    p.rows = rows; p.D = D; p.group = group; p.silu = gate_act == KDA_GATE_SILU; p.eps = eps;
    p.x_out = x_out; p.h = h;
    return kda::launch_block_norm(p, dt == KDA_F32 ? 0 : 1, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

size_t kda_block_norm_backward_workspace_bytes(int64_t rows, int32_t D, int32_t group) {
    if (rows < 0 || D < 1 || group < 1 || !supported_norm(D, group)) return 0;
    return (size_t)kda::block_norm_parts(rows, D) * 3 * D * sizeof(float);
}

int kda_block_norm_backward(const void* y, const float* w_post, const void* gate,
                            const void* x_out, const float* res_scale, const float* w_pre,
                            const void* dx_out, const void* dh, int64_t rows, int32_t D,
                            int32_t group, kda_dtype dt, int32_t gate_act, float eps, void* dy,
                            void* dgate, void* dx, float* dw_post, float* dres_scale,
                            float* dw_pre, void* workspace, size_t workspace_bytes,
                            void* stream) {
    const int bad = check_norm(y, w_post, rows, D, group, dt, gate_act, eps);
    if (bad != KDA_OK) return bad;
    if (rows > 0 && (!dy || (gate && !dgate) || (w_pre && (!x_out || !dh)) ||
                     (!dx_out && !w_pre))) {
        return KDA_ERR_INVALID_ARG;
    }
    if (!dw_post || (res_scale && !dres_scale) || (w_pre && !dw_pre) || (!gate && dgate) ||
        (!res_scale && dres_scale) || (!w_pre && (dw_pre || dh))) {
        return KDA_ERR_INVALID_ARG;
    }
    const size_t need = kda_block_norm_backward_workspace_bytes(rows, D, group);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const size_t n = (size_t)rows * D * elem_bytes(dt), nd = (size_t)D * sizeof(float);
    const size_t ng = (size_t)group * sizeof(float);
    const void* buf[15] = {y, gate, x_out, dx_out, dh, w_post, res_scale, w_pre,
                           dy, dgate, dx, dw_post, dres_scale, dw_pre, workspace};
    const size_t size[15] = {n, n, n, n, n, ng, nd, nd, n, n, n, ng, nd, nd, need};
    for (const void* b : buf) {
        if (!aligned(b, 16)) return KDA_ERR_ALIGNMENT;
    }
    for (int i = 8; i < 15; ++i) {      // no output, nor the workspace, on another buffer
        for (int j = 0; j < i; ++j) {
            if (overlaps(buf[i], size[i], buf[j], size[j])) return KDA_ERR_INVALID_ARG;
        }
    }
    kda::BlockNorm p;
    memset(&p, 0, sizeof(p));
    p.y = y; p.w_post = w_post; p.gate = gate; p.x = x_out; p.res_scale = res_scale;
    p.w_pre = w_pre; p.rows = rows; p.D = D; p.group = group;
    p.silu = gate_act == KDA_GATE_SILU; p.eps = eps;
    p.dx_out = dx_out; p.dh = dh; p.dy = dy; p.dgate = dgate; p.dx = dx;
    p.dw_post = dw_post; p.dres_scale = dres_scale; p.dw_pre = dw_pre;
    p.partial = static_cast<float*>(workspace);
    return kda::launch_block_norm_backward(p, dt == KDA_F32 ? 0 : 1,
                                           static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

}  // extern "C"
