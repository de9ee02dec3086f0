// kda_cache_plan.cu -- a step's bookkeeping on the device (kda_cache_plan in include/kda.h):
// three running sums over the requests (rows, returned blocks, taken blocks) and a look-up for
// each row.
//
// Bound by latency: one block of 1,024 threads does the requests, the sums in two passes
// because what is taken depends on how much all ended requests have returned; the rows, each of
// which finds its request by bisection of the row starts, are done by the same block up to 4,096
// of them, by many blocks in a second launch beyond.  256 requests of one token 5.4 us (two launches
// 8.4), 16 prompts of 109,824 tokens 13 us: the second launch, and one warp to each request's blocks,
// 32 of them at a time, each trip behind the one before (1,001 blocks of the longest prompt: 32 trips).
#include "../../include/kda.h"
#include "kda_cache.h"
#include "kda_follow.cuh"
#include "kda_seqlens.cuh"

namespace kda {
namespace {

constexpr int kThreads = 1024;
constexpr int kRowThreads = 256;
constexpr int kFewRows = 4096;       // that the one block does itself

struct Request {
    int64_t past, rows, have, want;
    bool bad, ends;
};

__device__ __forceinline__ Request request_of(const CachePlan& p, int i) {
    Request r;
    r.past = p.past[i];
    const int32_t fresh = p.fresh[i];
    r.bad = r.past < 0 || fresh < -1;
    r.rows = fresh > 0 ? fresh : 0;
    const int64_t round = (1 << p.block_log2) - 1;
    r.have = (r.past + round) >> p.block_log2;
    r.want = (r.past + r.rows + round) >> p.block_log2;
    r.ends = fresh == -1 && !r.bad && r.have <= p.width;
    return r;
}

// Running sum of x over the block's threads, this thread's own among them; *sum: all.
__device__ __forceinline__ int64_t running(int64_t x, int64_t* sum, int64_t (&warp)[33]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp[w] = x;
    __syncthreads();
    if (w == 0) {
        int64_t y = warp[lane];
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        warp[lane] = y;
    }
    __syncthreads();
    const int64_t before = w ? warp[w - 1] : 0;
    *sum = warp[31];
    __syncthreads();
    return before + x;
}

__device__ __forceinline__ int64_t clamped(int64_t x, int64_t hi) {
    return x < 0 ? 0 : (x > hi ? hi : x);
}

// Position and slot of row t; `starts`: the requests' first rows.
__device__ __forceinline__ void plan_row(const CachePlan& p, const int32_t* starts, int64_t t) {
    int32_t position = 0;
    int64_t slot = -1;
    if (t < starts[p.N]) {
        const int lo = last_start(starts, p.N, t);
        const int64_t at = (int64_t)p.past[lo] + t - starts[lo];
        position = (int32_t)(at < 0x7fffffff ? at : 0x7fffffff);
        if (p.status[lo] == KDA_PLAN_OK) {
            const int32_t b = p.table[(int64_t)lo * p.width + (at >> p.block_log2)];
            slot = ((int64_t)b << p.block_log2) + (at & ((1 << p.block_log2) - 1));
            if (b < 0 || slot > 0x7fffffff) slot = -1;
        }
    }
    p.positions[t] = position;
    p.slots[t] = (int32_t)slot;
}

__global__ void __launch_bounds__(kThreads, 1) plan_requests_kernel(CachePlan p, int rows_too) {
    __shared__ int64_t warp[33];
    __shared__ int64_t at[kThreads];
    __shared__ int32_t from[kThreads], count[kThreads], starts[kThreads + 1];
    let_follow();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t n_free = clamped(p.n_free[0], p.capacity);
    // rows, and the blocks of ended requests put back on the stack
    Request r = {};
    int64_t rows_before = 0, gone_before = 0, end = 0;
    for (int i0 = 0; i0 < p.N; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        r = Request();
        if (i < p.N) r = request_of(p, i);
        int64_t sum;
        end = rows_before + running(r.rows, &sum, warp);
        rows_before += sum;
        if (i < p.N) {
            p.cu[i + 1] = (int32_t)clamped(end, p.T);
            if (p.N <= kThreads) starts[i + 1] = (int32_t)clamped(end, p.T);
        }
        const int64_t gone = r.ends ? r.have : 0;
        if (!__syncthreads_or(gone > 0)) continue;
        at[threadIdx.x] = n_free + gone_before + running(gone, &sum, warp) - gone;
        count[threadIdx.x] = (int32_t)gone;
        gone_before += sum;
        __syncthreads();
        for (int k = w; k < kThreads && i0 + k < p.N; k += kThreads / 32) {
            const int32_t* row = p.table + (int64_t)(i0 + k) * p.width;
            for (int j = lane; j < count[k]; j += 32) {
                if (at[k] + j < p.capacity) p.free_blocks[at[k] + j] = row[j];
            }
        }
        __syncthreads();
    }
    const int64_t total = clamped(n_free + gone_before, p.capacity);
    // blocks taken from the stack's end, and what becomes of each request
    int64_t need_before = 0, taken = 0;
    rows_before = 0;
    for (int i0 = 0; i0 < p.N; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        int64_t sum;
        if (p.N > kThreads) {
            r = Request();
            if (i < p.N) r = request_of(p, i);
            end = rows_before + running(r.rows, &sum, warp);
            rows_before += sum;
        }
        int status = KDA_PLAN_OK;
        if (r.bad) {
            status = KDA_PLAN_BAD_LENGTH;
        } else if (r.want > p.width || r.past + r.rows > 0x7fffffff) {
            status = KDA_PLAN_TABLE;
        } else if (r.rows > 0 && end > p.T) {
            status = KDA_PLAN_ROWS;
        }
        const int64_t need = status == KDA_PLAN_OK && !r.ends ? r.want - r.have : 0;
        const int64_t upto = need_before + running(need, &sum, warp);
        const bool enough = need_before + sum <= total;
        need_before += sum;
        if (need > 0 && upto > total) status = KDA_PLAN_BLOCKS;
        const bool served = status == KDA_PLAN_OK;
        if (!enough) running(served ? need : 0, &sum, warp);
        taken += sum;
        at[threadIdx.x] = total - 1 - (upto - need);
        from[threadIdx.x] = (int32_t)r.have;
        count[threadIdx.x] = served ? (int32_t)need : 0;
        if (i < p.N) {
            p.status[i] = status;
            p.context[i] = served && !r.ends ? (int32_t)(r.past + r.rows) : 0;
        }
        __syncthreads();
        if (sum > 0) {
            for (int k = w; k < kThreads && i0 + k < p.N; k += kThreads / 32) {
                int32_t* row = p.table + (int64_t)(i0 + k) * p.width + from[k];
                for (int j = lane; j < count[k]; j += 32) row[j] = p.free_blocks[at[k] - j];
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        p.cu[0] = 0;
        starts[0] = 0;
        p.n_free_out[0] = (int32_t)(total - taken);
    }
    if (!rows_too) return;
    __syncthreads();
    for (int t = threadIdx.x; t < p.T; t += kThreads) {
        plan_row(p, p.N <= kThreads ? starts : p.cu, t);
    }
}

__global__ void __launch_bounds__(kRowThreads) plan_rows_kernel(CachePlan p) {
    wait_before();
    const int64_t t = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
    if (t < p.T) plan_row(p, p.cu, t);
}

}  // namespace

cudaError_t launch_cache_plan(const CachePlan& p, cudaStream_t stream) {
    const bool rows_too = p.T <= kFewRows;
    plan_requests_kernel<<<1, kThreads, 0, stream>>>(p, rows_too);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || rows_too) return err;
    return launch_follower(plan_rows_kernel, dim3((p.T + kRowThreads - 1) / kRowThreads),
                           dim3(kRowThreads), 0, stream, p);
}

}  // namespace kda
