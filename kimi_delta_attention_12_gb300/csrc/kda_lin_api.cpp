// kda_lin_api.cpp -- the C ABI of the decayed linear attention declared in
// include/kda.h: argument validation, workspace layout and launches on the
// caller's stream.  No allocation, no exceptions across the boundary.
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "kda_checks.h"
#include "kda_lin.h"

namespace {

using kda::aligned;
using kda::elem_bytes;
using kda::overlaps;
using kda::round_up;
using kda::supported_dim;

constexpr size_t kHeader = 256;   // status word
constexpr uint32_t kLinFlags = KDA_FLAG_RECURRENT;

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}

// Whether a pass runs on the tensor cores.
bool on_tensor_cores(int32_t d_k, int32_t d_v, kda_dtype dt, uint32_t flags, int32_t total_T) {
    return dt == KDA_BF16 && d_k == 128 && d_v == 128 && !(flags & KDA_FLAG_RECURRENT) &&
           total_T > 0;
}

// The tensor-core form works on a (sequence, head) pair of each of the `passes` it
// runs at once with one CTA an SM; the CUDA-core form with one CTA for each 32
// columns of dz, of which an SM takes two.  Its passes get segments for 8 CTAs an SM,
// the three of a backward for 3 each.  With 1, 2, 3, 4, 8, 16 CTAs, us, prefill: 5
// ragged sequences of 3,602 tokens, 8 heads, 64 x 128, fp32 186, 186, 122, 114, 106, 107;
// 4,096 tokens, 8 heads, 128 x 128, fp32 293, 169, 197, 173, 167, 167; 16,384, 4 heads 537,
// 285, 320, 326, 307, 325; 4,096, 32 heads, 64 x 64, bf16 430, 236, 243, 235, 221, 230.
// Backward of the same: 386, 419, 231, 243, 235, 235; 453, 460, 422, 437, 443, 443; 1,025,
// 812, 827, 842, 846, 868; 639, 605, 577, 590, 589, 617; 16 ragged sequences of 20,563
// tokens, 16 heads, 64 x 64, bf16 885, 886, 885, 885, 1,005, 1,058.
kda::LinCut cut_of(int32_t N, int32_t total_T, int32_t H, int32_t dz, int passes, bool tc) {
    return tc ? kda::lin_cut_tc(N, total_T, H, passes, sm_count())
              : kda::lin_cut(N, total_T, H, dz / 32, passes > 1 ? 3 : 8, sm_count());
}

size_t seg_state_bytes(int32_t total_T, int32_t H, int32_t dx, int32_t dz, int32_t seg_len) {
    return round_up((size_t)(total_T / seg_len) * H * dx * dz * sizeof(float), 256);
}

size_t state_bytes(int32_t N, int32_t H, int32_t d_k, int32_t d_v) {
    return (size_t)N * H * d_k * d_v * sizeof(float);
}

size_t decay_bytes(int32_t H) { return (size_t)H * sizeof(float); }
size_t seqlens_bytes(int32_t N) { return ((size_t)N + 1) * sizeof(int32_t); }

// Room for the segments' states of `passes` passes that run at once, whichever
// form a call's flags choose.
size_t segment_room(int32_t N, int32_t total_T, int32_t H, int32_t d_k, int32_t d_v, kda_dtype dt,
                    int passes) {
    const int32_t dz = d_k < d_v ? d_k : d_v;
    const size_t a =
        passes * seg_state_bytes(total_T, H, d_k, d_v, cut_of(N, total_T, H, dz, passes, false).seg_len);
    if (!on_tensor_cores(d_k, d_v, dt, 0, total_T)) return a;
    const size_t b = passes * seg_state_bytes(total_T, H, d_k, d_v,
                                              cut_of(N, total_T, H, dz, passes, true).seg_len);
    return a > b ? a : b;
}

bool bad_sizes(int32_t N, int32_t total_T, int32_t H) { return N < 1 || H < 1 || total_T < 0; }

}  // namespace

extern "C" {

size_t kda_lin_prefill_workspace_bytes(int32_t N, int32_t total_T, int32_t H, int32_t d_k,
                                       int32_t d_v, kda_dtype dt) {
    if (bad_sizes(N, total_T, H) || !supported_dim(d_k) || !supported_dim(d_v) ||
        (dt != KDA_F32 && dt != KDA_BF16)) {
        return 0;
    }
    // the states of the segments, and a copy of the initial states for a call
    // that updates them in place
    const size_t room = segment_room(N, total_T, H, d_k, d_v, dt, 1);
    return kHeader + room + (room > 0 ? round_up(state_bytes(N, H, d_k, d_v), 256) : 0);
}

int kda_lin_prefill(const void* q, const void* k, const void* v, const float* log_decay,
                    const float* initial_state, const int32_t* cu_seqlens,
                    const int32_t* cu_seqlens_host, int32_t N, int32_t total_T, int32_t H,
                    int32_t d_k, int32_t d_v, kda_dtype dt, float scale, uint32_t flags, void* o,
                    float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (!supported_dim(d_k) || !supported_dim(d_v)) return KDA_ERR_UNSUPPORTED;
    if (bad_sizes(N, total_T, H)) return KDA_ERR_INVALID_ARG;
    if ((flags & ~kLinFlags) != 0 || !isfinite(scale) || !log_decay) return KDA_ERR_INVALID_ARG;
    if (total_T > 0 && (!q || !k || !v || !o)) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && total_T % N != 0) return KDA_ERR_INVALID_ARG;
    if (cu_seqlens_host &&
        !kda::valid_host_seqlens(cu_seqlens_host, N, total_T, cu_seqlens == nullptr)) {
        return KDA_ERR_INVALID_ARG;
    }
    const size_t need = kda_lin_prefill_workspace_bytes(N, total_T, H, d_k, d_v, dt);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const size_t eb = elem_bytes(dt), nst = state_bytes(N, H, d_k, d_v);
    const size_t nqk = (size_t)total_T * H * d_k * eb, nv = (size_t)total_T * H * d_v * eb;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
        !aligned(log_decay, 4) || !aligned(initial_state, 16) || !aligned(final_state, 16) ||
        !aligned(cu_seqlens, 4) || !aligned(workspace, 256)) {
        return KDA_ERR_ALIGNMENT;
    }
    // o may not overlap an input; final_state only the initial one, whole
    const void* ins[6] = {q, k, v, initial_state, log_decay, cu_seqlens};
    const size_t nin[6] = {nqk, nqk, nv, nst, decay_bytes(H), seqlens_bytes(N)};
    const size_t used = need;
    for (int i = 0; i < 6; ++i) {
        if (overlaps(o, nv, ins[i], nin[i]) || overlaps(workspace, used, ins[i], nin[i])) {
            return KDA_ERR_INVALID_ARG;
        }
        if (overlaps(final_state, nst, ins[i], nin[i]) && !(i == 3 && ins[i] == final_state)) {
            return KDA_ERR_INVALID_ARG;
        }
    }
    if (overlaps(o, nv, final_state, nst) || overlaps(workspace, used, o, nv) ||
        overlaps(workspace, used, final_state, nst)) {
        return KDA_ERR_INVALID_ARG;
    }
    if (total_T == 0 && !final_state) return KDA_OK;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const bool tc = on_tensor_cores(d_k, d_v, dt, flags, total_T);
    kda::LinPass p;
    memset(&p, 0, sizeof(p));
    p.x = q; p.y = k; p.z = v; p.out = o;
    p.log_decay = log_decay;
    p.state_in = initial_state; p.state_out = final_state;
    p.cu_seqlens = cu_seqlens;
    p.status = reinterpret_cast<int32_t*>(ws);
    p.N = N; p.total_T = total_T; p.H = H; p.dx = d_k; p.dz = d_v;
    const kda::LinCut cut = cut_of(N, total_T, H, d_v, 1, tc);
    p.seg_len = cut.seg_len;
    p.lead = cut.lead;
    p.seg_states = reinterpret_cast<float*>(ws + kHeader);
    p.out_scale = scale; p.kv_scale = 1.0f;
    if (initial_state && initial_state == final_state && total_T / p.seg_len > 0) {
        // the last segment may write its state before the first has read it
        float* copy = reinterpret_cast<float*>(
            ws + kHeader + segment_room(N, total_T, H, d_k, d_v, dt, 1));
        if (cudaMemcpyAsync(copy, initial_state, nst, cudaMemcpyDeviceToDevice, s) !=
            cudaSuccess) {
            return KDA_ERR_CUDA;
        }
        p.state_in = copy;
    }
    const cudaError_t err = tc ? kda::launch_lin_pass_tc(&p, 1, s)
                               : kda::launch_lin_pass(&p, 1, dt == KDA_F32 ? 0 : 1, s);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_lin_decode_step(const void* q, const void* k, const void* v, const float* log_decay,
                        float* state, const int32_t* slots, int32_t pool_size, int32_t B,
                        int32_t H, int32_t d_k, int32_t d_v, kda_dtype dt, float scale, void* o,
                        void* stream) {
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (!supported_dim(d_k) || !supported_dim(d_v)) return KDA_ERR_UNSUPPORTED;
    if (B < 0 || H < 1 || pool_size < 0 || !isfinite(scale)) return KDA_ERR_INVALID_ARG;
    if (B == 0) return KDA_OK;
    if (!q || !k || !v || !log_decay || !state || !o) return KDA_ERR_INVALID_ARG;
    if (!slots && pool_size < B) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
        !aligned(state, 16) || !aligned(log_decay, 4) || !aligned(slots, 4)) {
        return KDA_ERR_ALIGNMENT;
    }
    const size_t eb = elem_bytes(dt), nqk = (size_t)B * H * d_k * eb,
                 nv = (size_t)B * H * d_v * eb, nst = state_bytes(pool_size, H, d_k, d_v);
    const void* ins[5] = {q, k, v, log_decay, slots};
    const size_t nin[5] = {nqk, nqk, nv, decay_bytes(H), (size_t)B * sizeof(int32_t)};
    for (int i = 0; i < 5; ++i) {
        if (overlaps(o, nv, ins[i], nin[i]) || overlaps(state, nst, ins[i], nin[i])) {
            return KDA_ERR_INVALID_ARG;
        }
    }
    if (overlaps(o, nv, state, nst)) return KDA_ERR_INVALID_ARG;
    kda::LinDecode p;
    p.q = q; p.k = k; p.v = v; p.log_decay = log_decay; p.state = state; p.slots = slots; p.o = o;
    p.pool_size = pool_size; p.B = B; p.H = H; p.scale = scale;
    return kda::launch_lin_decode(p, d_k, d_v, dt == KDA_F32 ? 0 : 1,
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

// The three passes run at once, each with segments' states of its own.
size_t kda_lin_backward_workspace_bytes(int32_t N, int32_t total_T, int32_t H, int32_t d_k,
                                        int32_t d_v, kda_dtype dt) {
    if (bad_sizes(N, total_T, H) || !supported_dim(d_k) || !supported_dim(d_v) ||
        (dt != KDA_F32 && dt != KDA_BF16)) {
        return 0;
    }
    return kHeader + segment_room(N, total_T, H, d_k, d_v, dt, 3);
}

int kda_lin_backward(const void* q, const void* k, const void* v, const float* log_decay,
                     const float* initial_state, const int32_t* cu_seqlens,
                     const int32_t* cu_seqlens_host, int32_t N, int32_t total_T, int32_t H,
                     int32_t d_k, int32_t d_v, kda_dtype dt, float scale, uint32_t flags,
                     const void* dO, const float* dS_final, void* dq, void* dk, void* dv,
                     float* dS0, void* workspace, size_t workspace_bytes, void* stream) {
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (!supported_dim(d_k) || !supported_dim(d_v)) return KDA_ERR_UNSUPPORTED;
    if (bad_sizes(N, total_T, H)) return KDA_ERR_INVALID_ARG;
    if ((flags & ~kLinFlags) != 0 || !isfinite(scale) || !log_decay) return KDA_ERR_INVALID_ARG;
    if (total_T > 0 && (!q || !k || !v || !dO || !dq || !dk || !dv)) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && total_T % N != 0) return KDA_ERR_INVALID_ARG;
    if (cu_seqlens_host &&
        !kda::valid_host_seqlens(cu_seqlens_host, N, total_T, cu_seqlens == nullptr)) {
        return KDA_ERR_INVALID_ARG;
    }
    const size_t need = kda_lin_backward_workspace_bytes(N, total_T, H, d_k, d_v, dt);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const void* bufs[13] = {log_decay, cu_seqlens, q, k, v, dO, initial_state, dS_final,
                            dq, dk, dv, dS0, workspace};
    for (int i = 2; i < 12; ++i) {
        if (!aligned(bufs[i], 16)) return KDA_ERR_ALIGNMENT;
    }
    if (!aligned(log_decay, 4) || !aligned(cu_seqlens, 4) || !aligned(workspace, 256)) {
        return KDA_ERR_ALIGNMENT;
    }
    const size_t eb = elem_bytes(dt), nst = state_bytes(N, H, d_k, d_v);
    const size_t nqk = (size_t)total_T * H * d_k * eb, nv = (size_t)total_T * H * d_v * eb;
    const size_t size[13] = {decay_bytes(H), seqlens_bytes(N), nqk, nqk, nv, nv, nst, nst,
                             nqk, nqk, nv, nst, need};
    for (int i = 8; i < 13; ++i) {      // no output, nor the workspace, on another buffer
        for (int j = 0; j < i; ++j) {
            if (overlaps(bufs[i], size[i], bufs[j], size[j])) return KDA_ERR_INVALID_ARG;
        }
    }
    if (total_T == 0 && !dS0) return KDA_OK;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const bool tc = on_tensor_cores(d_k, d_v, dt, flags, total_T);
    kda::LinPass pass[3];
    memset(pass, 0, sizeof(pass));
    for (kda::LinPass& p : pass) {
        p.log_decay = log_decay;
        p.cu_seqlens = cu_seqlens;
        p.status = reinterpret_cast<int32_t*>(ws);
        p.N = N; p.total_T = total_T; p.H = H;
    }
    // dq_t = scale S_t dO_t: forward in time with the turned state
    kda::LinPass& a = pass[0];
    a.x = dO; a.y = v; a.z = k; a.out = dq; a.dx = d_v; a.dz = d_k;
    a.state_in = initial_state; a.state_in_turned = 1;
    a.out_scale = scale; a.kv_scale = 1.0f;
    // dk_t = G_t v_t, G_t = scale q_t dO_t^T + a G_{t+1}: from the ends
    kda::LinPass& b = pass[1];
    b.x = v; b.y = dO; b.z = q; b.out = dk; b.dx = d_v; b.dz = d_k;
    b.state_in = dS_final; b.state_in_turned = 1;
    b.reverse = 1; b.out_scale = 1.0f; b.kv_scale = scale;
    // dv_t = G_t^T k_t; the state it ends with is dS_0
    kda::LinPass& c = pass[2];
    c.x = k; c.y = q; c.z = dO; c.out = dv; c.dx = d_k; c.dz = d_v;
    c.state_in = dS_final; c.state_out = dS0;
    c.reverse = 1; c.out_scale = 1.0f; c.kv_scale = scale;
    float* states = reinterpret_cast<float*>(ws + kHeader);
    if (tc) {
        const kda::LinCut cut = cut_of(N, total_T, H, d_v, 3, true);
        for (int i = 0; i < 3; ++i) {
            pass[i].seg_len = cut.seg_len;
            pass[i].lead = cut.lead;
            pass[i].seg_states =
                states + i * (seg_state_bytes(total_T, H, d_k, d_v, cut.seg_len) / sizeof(float));
        }
        return kda::launch_lin_pass_tc(pass, 3, s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    }
    for (kda::LinPass& p : pass) {
        p.seg_len = cut_of(N, total_T, H, p.dz, 3, false).seg_len;
        p.seg_states = states;
        states += seg_state_bytes(total_T, H, d_k, d_v, p.seg_len) / sizeof(float);
    }
    // (without tokens only the state is handed on)
    const cudaError_t err = total_T > 0 ? kda::launch_lin_pass(pass, 3, dt == KDA_F32 ? 0 : 1, s)
                                        : kda::launch_lin_pass(&c, 1, dt == KDA_F32 ? 0 : 1, s);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
