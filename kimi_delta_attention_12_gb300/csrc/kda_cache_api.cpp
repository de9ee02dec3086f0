// kda_cache_api.cpp -- the C ABI of the rotary positions and of the paged 8-bit cache
// declared in include/kda.h: argument validation and launches on the caller's stream.  No
// allocation, no exceptions across the boundary.
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "kda_cache.h"
#include "kda_checks.h"

namespace {

using kda::aligned;
using kda::elem_bytes;
using kda::overlaps;
using kda::round_up;
using kda::supported_dim;

constexpr size_t kHeader = 256;   // status word
constexpr int32_t kMaxRotaryDim = 512;
constexpr float kMostFrequency = 0x1p20f;   // that kda_rotary is made for
constexpr int32_t kMaxGroup = 64;
constexpr int32_t kMostRows = 0x7fff0000;   // whole tiles of rows stay within 32 bits
constexpr uint32_t kRotaryFlags = KDA_FLAG_ROTARY_INTERLEAVED | KDA_FLAG_ROTARY_INVERSE;

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}

// Rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void* p;
    int64_t n;
    size_t stride, width;
    size_t span() const { return n > 0 ? (size_t)(n - 1) * stride + width : 0; }
};

// Whether two sets of rows share a byte.  Rows of one stride that lie beside each other
// (parts of one wider buffer) do not.
bool rows_overlap(const Rows& a, const Rows& b) {
    if (!overlaps(a.p, a.span(), b.p, b.span())) return false;
    if (a.stride != b.stride) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const size_t s = a.stride, ahead = y >= x ? (y - x) % s : (s - (x - y) % s) % s;
    return !(ahead >= a.width && ahead + b.width <= s);
}

// A row stride in elements: at least a row, whole 16-byte vectors.
bool good_stride(int64_t stride, int64_t width, kda_dtype dt) {
    return stride >= width && stride < ((int64_t)1 << 40) && stride * elem_bytes(dt) % 16 == 0;
}

int log2_of_block(int32_t block) {
    return block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : block == 128 ? 7 : -1;
}

size_t attention_room(int32_t T, int32_t max_new, int32_t Hq, int32_t Hkv, int32_t d,
                      kda_dtype dt, int sms) {
    return kHeader + round_up(kda::cache_attention_room(Hkv, Hq / Hkv, T, max_new, d,
                                                        dt == KDA_F32 ? 0 : 1, sms), 256);
}

bool good_type(kda_dtype dt) { return dt == KDA_F32 || dt == KDA_BF16; }

// What the cache's calls check alike; KDA_OK, or the error.
int check_cache(const void* k_cache, const void* v_cache, const float* k_scale,
                const float* v_scale, int32_t num_blocks, int32_t block, int32_t heads, int32_t d,
                kda_dtype dt) {
    if (!good_type(dt) || !supported_dim(d) || log2_of_block(block) < 0) return KDA_ERR_UNSUPPORTED;
    if (heads < 1 || heads > 65535 || num_blocks < 1) return KDA_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * block > 0x7fffffff) return KDA_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !k_scale || !v_scale) return KDA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4)) {
        return KDA_ERR_ALIGNMENT;
    }
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_rotary_frequencies(int32_t rot, double base, kda_rotary_scaling scaling, double factor,
                           double original_length, double fast, double slow, float* inv_freq,
                           float* magnitude) {
    if (rot < 2 || rot > 65536 || rot % 2 != 0 || !inv_freq || !magnitude) {
        return KDA_ERR_INVALID_ARG;
    }
    const bool linear = scaling == KDA_ROTARY_LINEAR, parts = scaling == KDA_ROTARY_BY_PARTS;
    if (!(linear || parts || scaling == KDA_ROTARY_PLAIN)) return KDA_ERR_INVALID_ARG;
    if (!isfinite(base) || base <= 0.0) return KDA_ERR_INVALID_ARG;
    if ((linear || parts) && (!isfinite(factor) || factor <= 0.0)) return KDA_ERR_INVALID_ARG;
    if (parts && (!isfinite(original_length) || original_length <= 0.0 || !isfinite(fast) ||
                  !isfinite(slow) || slow <= 0.0 || fast <= slow)) {
        return KDA_ERR_INVALID_ARG;
    }
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    auto frequency = [&](int32_t j) {
        double f = pow(base, -2.0 * j / rot);
        if (linear) {
            f /= factor;
        } else if (parts) {
            const double turns = original_length * f / kTwoPi;
            double w = (turns - slow) / (fast - slow);
            w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
            f = f * w + f / factor * (1.0 - w);
        }
        return f;
    };
    for (int32_t j = 0; j < rot / 2; ++j) {
        if (!((float)frequency(j) < kMostFrequency)) return KDA_ERR_INVALID_ARG;
    }
    for (int32_t j = 0; j < rot / 2; ++j) inv_freq[j] = (float)frequency(j);
    // (a factor below 1 lengthens nothing, and far below it the logarithm would turn pairs around)
    *magnitude = parts && factor > 1.0 ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return KDA_OK;
}

int kda_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
               const int32_t* positions, const float* inv_freq, int64_t T, int32_t Hq, int32_t Hk,
               int32_t d, int32_t rot, int32_t first, kda_dtype dt, uint32_t flags,
               float magnitude, void* q_out, int64_t q_out_stride, void* k_out,
               int64_t k_out_stride, void* stream) {
    if (!good_type(dt)) return KDA_ERR_UNSUPPORTED;
    if (d < 8 || d > kMaxRotaryDim || d % 8 != 0 || rot < 16 || rot % 16 != 0 || first < 0 ||
        first % 8 != 0 || rot > d || first > d - rot) {
        return KDA_ERR_UNSUPPORTED;
    }
    if (T < 0 || T > ((int64_t)1 << 31) || Hq < 1 || Hk < 0 || Hq > 65535 || Hk > 65535 ||
        (flags & ~kRotaryFlags) != 0 || !isfinite(magnitude) || !inv_freq) {
        return KDA_ERR_INVALID_ARG;
    }
    if (T > 0 && (!q || !q_out || !positions || (Hk > 0) != (k != nullptr) ||
                  (Hk > 0) != (k_out != nullptr))) {
        return KDA_ERR_INVALID_ARG;
    }
    const int64_t nq = (int64_t)Hq * d, nk = (int64_t)Hk * d;
    if (!good_stride(q_stride, nq, dt) || !good_stride(q_out_stride, nq, dt) ||
        (Hk > 0 && (!good_stride(k_stride, nk, dt) || !good_stride(k_out_stride, nk, dt)))) {
        return KDA_ERR_INVALID_ARG;
    }
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
        !aligned(positions, 4) || !aligned(inv_freq, 4)) {
        return KDA_ERR_ALIGNMENT;
    }
    const size_t eb = elem_bytes(dt);
    const Rows in[2] = {{q, T, (size_t)q_stride * eb, (size_t)nq * eb},
                        {k, Hk > 0 ? T : 0, (size_t)k_stride * eb, (size_t)nk * eb}};
    const Rows out[2] = {{q_out, T, (size_t)q_out_stride * eb, (size_t)nq * eb},
                         {k_out, Hk > 0 ? T : 0, (size_t)k_out_stride * eb, (size_t)nk * eb}};
    for (int o = 0; o < 2; ++o) {
        for (int i = 0; i < 2; ++i) {
            const bool itself = i == o && out[o].p == in[i].p &&
                                (T <= 1 || out[o].stride == in[i].stride);
            if (!itself && rows_overlap(out[o], in[i])) return KDA_ERR_INVALID_ARG;
        }
        if (overlaps(out[o].p, out[o].span(), positions, (size_t)T * 4) ||
            overlaps(out[o].p, out[o].span(), inv_freq, (size_t)rot * 2)) {
            return KDA_ERR_INVALID_ARG;
        }
    }
    if (rows_overlap(out[0], out[1])) return KDA_ERR_INVALID_ARG;
    if (T == 0) return KDA_OK;
    kda::Rotary p;
    memset(&p, 0, sizeof(p));
    p.x[0] = q; p.x[1] = k; p.out[0] = q_out; p.out[1] = k_out;
    p.stride[0] = q_stride; p.stride[1] = k_stride;
    p.out_stride[0] = q_out_stride; p.out_stride[1] = k_out_stride;
    p.heads[0] = Hq; p.heads[1] = Hk;
    p.positions = positions; p.inv_freq = inv_freq;
    p.T = T; p.d = d; p.rot = rot; p.first = first;
    p.interleaved = (flags & KDA_FLAG_ROTARY_INTERLEAVED) != 0;
    p.inverse = (flags & KDA_FLAG_ROTARY_INVERSE) != 0;
    p.magnitude = magnitude;
    return kda::launch_rotary(p, dt == KDA_F32 ? 0 : 1, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

int kda_cache_plan(const int32_t* past, const int32_t* new_tokens, int32_t N, int32_t* block_table,
                   int32_t table_width, int32_t* free_blocks, int32_t free_capacity,
                   const int32_t* n_free, int32_t* n_free_out, int32_t block, int32_t T,
                   int32_t* cu_seqlens, int32_t* context_lens, int32_t* positions, int32_t* slots,
                   int32_t* status, void* stream) {
    if (log2_of_block(block) < 0 || N > kMostRows || T > kMostRows) return KDA_ERR_UNSUPPORTED;
    if (N < 1 || T < 0 || table_width < 1 || free_capacity < 1 || !past || !new_tokens ||
        !block_table || !free_blocks || !n_free || !n_free_out || !cu_seqlens || !context_lens ||
        !status || (T > 0 && (!positions || !slots))) {
        return KDA_ERR_INVALID_ARG;
    }
    const size_t n = (size_t)N * 4, rows = (size_t)T * 4;
    const void* buf[11] = {past, new_tokens, n_free, block_table, free_blocks, n_free_out,
                           cu_seqlens, context_lens, positions, slots, status};
    const size_t size[11] = {n, n, 4, n * (size_t)table_width, (size_t)free_capacity * 4, 4,
                             n + 4, n, rows, rows, n};
    for (const void* b : buf) {
        if (!aligned(b, 4)) return KDA_ERR_ALIGNMENT;
    }
    for (int i = 3; i < 11; ++i) {      // no output on another buffer, but n_free on itself
        for (int j = 0; j < i; ++j) {
            if (overlaps(buf[i], size[i], buf[j], size[j]) &&
                !(i == 5 && j == 2 && buf[i] == buf[j])) {
                return KDA_ERR_INVALID_ARG;
            }
        }
    }
    kda::CachePlan p;
    memset(&p, 0, sizeof(p));
    p.past = past; p.fresh = new_tokens; p.N = N; p.table = block_table; p.width = table_width;
    p.free_blocks = free_blocks; p.capacity = free_capacity; p.n_free = n_free;
    p.n_free_out = n_free_out; p.block_log2 = log2_of_block(block); p.T = T; p.cu = cu_seqlens;
    p.context = context_lens; p.positions = positions; p.slots = slots; p.status = status;
    return kda::launch_cache_plan(p, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

int kda_cache_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                    const int32_t* slots, int32_t T, int32_t Hkv, int32_t d, kda_dtype dt,
                    void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                    int32_t num_blocks, int32_t block, void* stream) {
    const int bad = check_cache(k_cache, v_cache, k_scale, v_scale, num_blocks, block, Hkv, d, dt);
    if (bad != KDA_OK) return bad;
    if (T < 0 || (T > 0 && (!k || !v || !slots))) return KDA_ERR_INVALID_ARG;
    if (T > kMostRows) return KDA_ERR_UNSUPPORTED;
    const int64_t width = (int64_t)Hkv * d;
    if (!good_stride(k_stride, width, dt) || !good_stride(v_stride, width, dt)) {
        return KDA_ERR_INVALID_ARG;
    }
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return KDA_ERR_ALIGNMENT;
    const size_t eb = elem_bytes(dt);
    const Rows kr = {k, T, (size_t)k_stride * eb, (size_t)width * eb};
    const Rows vr = {v, T, (size_t)v_stride * eb, (size_t)width * eb};
    const size_t pool = (size_t)num_blocks * block * width, scales = (size_t)num_blocks * Hkv * 4;
    const void* buf[7] = {k, v, slots, k_cache, v_cache, k_scale, v_scale};
    const size_t size[7] = {kr.span(), vr.span(), (size_t)T * 4, pool, pool, scales, scales};
    for (int i = 3; i < 7; ++i) {
        for (int j = 0; j < i; ++j) {
            if (overlaps(buf[i], size[i], buf[j], size[j])) return KDA_ERR_INVALID_ARG;
        }
    }
    if (T == 0) return KDA_OK;
    kda::CacheWrite p;
    memset(&p, 0, sizeof(p));
    p.x[0] = k; p.x[1] = v; p.stride[0] = k_stride; p.stride[1] = v_stride;
    p.cache[0] = static_cast<uint8_t*>(k_cache); p.cache[1] = static_cast<uint8_t*>(v_cache);
    p.scale[0] = k_scale; p.scale[1] = v_scale;
    p.slots = slots; p.T = T; p.heads = Hkv; p.d = d; p.num_blocks = num_blocks;
    p.block_log2 = log2_of_block(block);
    return kda::launch_cache_write(p, dt == KDA_F32 ? 0 : 1, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

size_t kda_cache_attention_workspace_bytes(int32_t T, int32_t max_new, int32_t Hq, int32_t Hkv,
                                           int32_t d, kda_dtype dt) {
    if (T < 0 || max_new < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > kMaxGroup ||
        !supported_dim(d) || !good_type(dt)) {
        return 0;
    }
    return attention_room(T, max_new, Hq, Hkv, d, dt, sm_count());
}

int kda_cache_attention(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                        const float* k_scale, const float* v_scale, int32_t num_blocks,
                        int32_t block, const int32_t* block_table, int32_t table_width,
                        const int32_t* context_lens, const int32_t* cu_seqlens, int32_t N,
                        int32_t T, int32_t max_new, int32_t Hq, int32_t Hkv, int32_t d,
                        kda_dtype dt, float scale, void* o, void* workspace,
                        size_t workspace_bytes, void* stream) {
    const int bad = check_cache(k_cache, v_cache, k_scale, v_scale, num_blocks, block, Hkv, d, dt);
    if (bad != KDA_OK) return bad;
    if (Hq < Hkv || Hq % Hkv != 0 || N < 1 || T < 0 || max_new < 0 || table_width < 1 ||
        !isfinite(scale) || (!cu_seqlens && T != N)) {
        return KDA_ERR_INVALID_ARG;
    }
    const int32_t group = Hq / Hkv;
    if (group > kMaxGroup || (int64_t)T * group > kMostRows || N > kMostRows) {
        return KDA_ERR_UNSUPPORTED;
    }
    if (!block_table || !context_lens || (T > 0 && (!q || !o))) return KDA_ERR_INVALID_ARG;
    const int64_t width = (int64_t)Hq * d;
    if (!good_stride(q_stride, width, dt)) return KDA_ERR_INVALID_ARG;
    const int sms = sm_count();
    const size_t need = attention_room(T, max_new, Hq, Hkv, d, dt, sms);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(block_table, 4) ||
        !aligned(context_lens, 4) || !aligned(cu_seqlens, 4) || !aligned(workspace, 256)) {
        return KDA_ERR_ALIGNMENT;
    }
    const size_t eb = elem_bytes(dt);
    const Rows qr = {q, T, (size_t)q_stride * eb, (size_t)width * eb};
    const size_t pool = (size_t)num_blocks * block * Hkv * d, scales = (size_t)num_blocks * Hkv * 4;
    const size_t out = (size_t)T * width * eb;
    const void* in[8] = {q, k_cache, v_cache, k_scale, v_scale, block_table, context_lens,
                         cu_seqlens};
    const size_t size[8] = {qr.span(), pool, pool, scales, scales, (size_t)N * table_width * 4,
                            (size_t)N * 4, (size_t)N * 4 + 4};
    for (int i = 0; i < 8; ++i) {
        if (overlaps(o, out, in[i], size[i]) || overlaps(workspace, need, in[i], size[i])) {
            return KDA_ERR_INVALID_ARG;
        }
    }
    if (overlaps(o, out, workspace, need)) return KDA_ERR_INVALID_ARG;
    if (T == 0) return KDA_OK;
    if (sms < 1) return KDA_ERR_CUDA;
    kda::CacheAttention p;
    memset(&p, 0, sizeof(p));
    p.q = q; p.q_stride = q_stride;
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = k_scale; p.v_scale = v_scale; p.num_blocks = num_blocks;
    p.block_log2 = log2_of_block(block); p.table = block_table; p.width = table_width;
    p.context = context_lens; p.cu = cu_seqlens; p.N = N; p.T = T; p.max_new = max_new;
    p.heads = Hkv; p.group = group; p.d = d; p.scale = scale; p.o = o;
    p.status = static_cast<int32_t*>(workspace);
    p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeader);
    return kda::launch_cache_attention(p, dt == KDA_F32 ? 0 : 1, sms,
                                       static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

}  // extern "C"
