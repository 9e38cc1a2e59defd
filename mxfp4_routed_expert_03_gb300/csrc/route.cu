// Routing: per-token top-k with softmax weights (K1) and the per-expert route
// plan (K2: histogram, exclusive scan, stable counting-sort scatter).
//
// Each token selects top_k of n_experts experts (MoonTail, intro; Moonshine
// README, "How the engine works"). All rows selecting each expert are then
// grouped and only the experts with rows are touched (Moonshine README,
// "How the engine works", prefill paragraph; Moonshine GitHub README,
// "Prefill"). Order: descending logit, ties to the lower expert index; the
// weights are the softmax over the selected logits. The plan orders the flat
// indices t*k+j by (expert, flat index), so it is unique and bit-exact.
#include "route.cuh"

using namespace moe_route;

// ---------------------------------------------------------------------------
// Small batches: one CTA does top-k, histogram, scan and the stable scatter.
// 512 threads (16 warps), one warp per token (warp_topk). (A 1024-thread
// block would cap a thread at 64 registers and push the keys to local
// memory.) The scans take two experts per thread.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanSmallThreads) moe_plan_small_kernel(
    int T, int E, int k, const float *__restrict__ logits, moe_plan_buf p, int *status) {
    __shared__ PlanSmall s;  // T <= 64 tokens, k <= 32: the selections stay in shared memory
    int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    grid_dep_wait();    // the logits may come from the previous kernel
    grid_dep_launch();
    plan_small_init(s);
    bool nan_seen = false;
    for (int t = wid; t < T; t += kPlanSmallWarps) {
        int my_e;
        float my_v;
        warp_topk<true>(logits + (int64_t)t * E, E, k, lane, my_e, my_v, nan_seen, s.scr[wid]);
        plan_small_put(s, t, k, lane, my_e, warp_select_weight(my_v, k, lane), p.topk_idx, p.topk_w);
    }
    plan_small_finish(s, T, E, k, nan_seen, p, status);
}

// ---------------------------------------------------------------------------
// Large batches: four kernels.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) moe_topk_kernel(int T, int E, int k,
                                                       const float *__restrict__ logits,
                                                       int32_t *topk_idx, float *topk_w,
                                                       int *status) {
    __shared__ uint2 s_scratch[8][MOE_MAX_TOPK];
    int lane = threadIdx.x & 31;
    int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= T) return;
    int my_e;
    float my_v;
    bool nan_seen = false;
    warp_topk<false>(logits + (int64_t)t * E, E, k, lane, my_e, my_v, nan_seen,
                     s_scratch[threadIdx.x >> 5]);
    float w = warp_select_weight(my_v, k, lane);
    if (lane < k) {
        topk_idx[(int64_t)t * k + lane] = my_e;
        topk_w[(int64_t)t * k + lane] = w;
    }
    if (__any_sync(FULL_MASK, nan_seen) && lane == 0) moe_flag(status, MOE_ERR_NAN_LOGIT);
}

// chunk_counts[c][e]: rows of expert e among the 32 tokens of chunk c; a block
// per chunk (see plan_chunk_mask).
__global__ void __launch_bounds__(256) moe_plan_count_kernel(int T, int E, int k,
                                                             const int32_t *__restrict__ idx,
                                                             int32_t *chunk_counts, int *status) {
    __shared__ uint32_t s_mask[MOE_MAX_EXPERTS];
    plan_chunk_mask(s_mask, T, E, k, blockIdx.x, idx, status);
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        chunk_counts[(int64_t)blockIdx.x * E + e] = __popc(s_mask[e]);
}

// Per expert, chunk_counts to exclusive prefixes over the chunks (in place) and
// their total to counts. A block takes 32 experts (a 128-byte line per chunk),
// each warp a range of chunks: its sum, the ranges' prefixes, then the chunks'.
__global__ void __launch_bounds__(1024) moe_plan_scan_kernel(int E, int nchunks, int32_t *chunk_counts,
                                                             int32_t *counts) {
    __shared__ int s_sum[32][33];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    grid_dep_wait();
    grid_dep_launch();
    const int per = (nchunks + 31) / 32, c0 = wid * per, c1 = min(c0 + per, nchunks);
    int sum = 0;
    if (e < E) {
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += chunk_counts[(int64_t)c * E + e];
    }
    s_sum[wid][lane] = sum;
    __syncthreads();
    int run = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
        if (w == wid) run = total;
        total += s_sum[w][lane];
    }
    if (e >= E) return;
    for (int c = c0; c < c1; c += 8) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < c1 ? chunk_counts[(int64_t)(c + i) * E + e] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i < c1) chunk_counts[(int64_t)(c + i) * E + e] = run;
            run += v[i];
        }
    }
    if (wid == 0) counts[e] = total;
}

// A block per chunk: position of every entry = offsets[e] (scanned from counts
// by each block) + rows of e in earlier chunks + tokens of the chunk before it
// that chose e. Block 0 writes offsets and active.
__global__ void __launch_bounds__(256) moe_plan_scatter_kernel(int T, int E, int k,
                                                               const int32_t *__restrict__ idx,
                                                               const int32_t *__restrict__ chunk_base,
                                                               moe_plan_buf p, int *status) {
    __shared__ uint32_t s_mask[MOE_MAX_EXPERTS];
    __shared__ int s_off[MOE_MAX_EXPERTS], s_tot[33];
    static_assert(MOE_MAX_EXPERTS == 4 * 256, "four experts per thread in the scans");
    grid_dep_wait();
    grid_dep_launch();
    const int e0 = 4 * threadIdx.x, c = blockIdx.x;
    int n[4], sum = 0, used = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        n[i] = e0 + i < E ? p.counts[e0 + i] : 0;
        sum += n[i];
        used += n[i] > 0 ? 1 : 0;
    }
    plan_chunk_mask(s_mask, T, E, k, c, idx, status);
    int off = block_exclusive_scan<8>(sum, s_tot, total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s_off[e0 + i] = off;
        if (c == 0 && e0 + i < E) p.offsets[e0 + i] = off;
        off += n[i];
    }
    if (c == 0) {
        int at = block_exclusive_scan<8>(used, s_tot, total);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n[i] > 0) p.active[1 + at++] = e0 + i;
        if (threadIdx.x == 0) {
            p.offsets[E] = T * k;
            p.active[0] = total;
        }
    }
    __syncthreads();
    const int64_t f0 = (int64_t)c * MOE_PLAN_CHUNK * k;
    const int nf = (int)(min((int64_t)(c + 1) * MOE_PLAN_CHUNK, (int64_t)T) * k - f0);
    for (int i = threadIdx.x; i < nf; i += 256) {
        const int e = idx[f0 + i];
        if (e < 0 || e >= E) continue;  // (flagged above)
        const int pos = s_off[e] + chunk_base[(int64_t)c * E + e] +
                        __popc(s_mask[e] & ((1u << (i / k)) - 1u));
        p.perm[pos] = (int32_t)(f0 + i);
        p.inv[f0 + i] = pos;
    }
}

// ---------------------------------------------------------------------------
// Host launchers.
// ---------------------------------------------------------------------------
size_t moe_plan_ws_bytes(int T, int E) {
    if (T <= 0 || moe_plan_is_small(T)) return 0;
    int nchunks = (T + MOE_PLAN_CHUNK - 1) / MOE_PLAN_CHUNK;
    return (size_t)nchunks * E * sizeof(int32_t);
}

cudaError_t moe_launch_plan(int T, int E, int k, const float *logits, const moe_plan_buf *p,
                            void *ws, int *status, cudaStream_t st) {
    if (moe_plan_is_small(T)) {
        return launch_pdl(moe_plan_small_kernel, dim3(1), dim3(kPlanSmallThreads), 0, st,
                          T, E, k, logits, *p, status);
    }
    moe_topk_kernel<<<(T + 7) / 8, 256, 0, st>>>(T, E, k, logits, p->topk_idx, p->topk_w, status);
    return moe_launch_plan_build(T, E, k, false, p, ws, status, st);
}

cudaError_t moe_plan_setup() {
    cudaError_t err = set_kernel((const void *)moe_plan_scan_kernel);
    if (err == cudaSuccess) err = set_kernel((const void *)moe_plan_scatter_kernel);
    return err != cudaSuccess ? err : moe_plan_scored_setup();
}

cudaError_t moe_launch_plan_build(int T, int E, int k, bool counted, const moe_plan_buf *p, void *ws,
                                  int *status, cudaStream_t st) {
    const int nchunks = (T + MOE_PLAN_CHUNK - 1) / MOE_PLAN_CHUNK;
    int32_t *chunk = (int32_t *)ws;
    if (!counted)
        moe_plan_count_kernel<<<nchunks, 256, 0, st>>>(T, E, k, p->topk_idx, chunk, status);
    cudaError_t err = cudaGetLastError();
    if (err == cudaSuccess)
        err = launch_pdl_ready(moe_plan_scan_kernel, dim3((E + 31) / 32), dim3(1024), 0, st, E, nchunks, chunk,
                         p->counts);
    if (err == cudaSuccess)
        err = launch_pdl_ready(moe_plan_scatter_kernel, dim3(nchunks), dim3(256), 0, st, T, E, k,
                         (const int32_t *)p->topk_idx, (const int32_t *)chunk, *p, status);
    return err;
}
