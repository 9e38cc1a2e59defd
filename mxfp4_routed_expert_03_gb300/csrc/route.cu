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

// chunk_counts[c][e]: rows of expert e among tokens [c*CH, (c+1)*CH).
__global__ void __launch_bounds__(256) moe_plan_count_kernel(int T, int E, int k, int CH,
                                                             const int32_t *__restrict__ idx,
                                                             int32_t *chunk_counts, int *status) {
    extern __shared__ int s_hist[];  // 8 warps x E
    int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int c = blockIdx.x * 8 + wid;
    int nchunks = (T + CH - 1) / CH;
    int *h = s_hist + wid * E;
    for (int e = lane; e < E; e += 32) h[e] = 0;
    __syncwarp();
    if (c < nchunks) {
        int64_t f0 = (int64_t)c * CH * k;
        int64_t f1 = min((int64_t)(c + 1) * CH, (int64_t)T) * k;
        for (int64_t f = f0 + lane; f < f1; f += 32) {
            int e = idx[f];
            if (e >= 0 && e < E) atomicAdd(&h[e], 1);
            else moe_flag(status, MOE_ERR_BAD_INDEX);
        }
        __syncwarp();
        for (int e = lane; e < E; e += 32) chunk_counts[(int64_t)c * E + e] = h[e];
    }
}

// Column scan of chunk_counts (in place -> chunk bases), counts, offsets, active.
__global__ void __launch_bounds__(1024) moe_plan_scan_kernel(int T, int E, int k, int nchunks,
                                                             int32_t *chunk_counts,
                                                             int32_t *counts, int32_t *offsets,
                                                             int32_t *active) {
    __shared__ int s_tot[33];
    int e = threadIdx.x;
    int run = 0;
    if (e < E) {
        for (int c = 0; c < nchunks; ++c) {
            int v = chunk_counts[(int64_t)c * E + e];
            chunk_counts[(int64_t)c * E + e] = run;
            run += v;
        }
    }
    int total;
    int off = block_exclusive_scan<32>(run, s_tot, total);
    int a = block_exclusive_scan<32>(run > 0 ? 1 : 0, s_tot, total);
    if (e < E) {
        counts[e] = run;
        offsets[e] = off;
        if (run > 0) active[1 + a] = e;
    }
    if (e == 0) {
        offsets[E] = T * k;
        active[0] = total;
    }
}

__global__ void __launch_bounds__(256) moe_plan_scatter_kernel(int T, int E, int k, int CH,
                                                               const int32_t *__restrict__ idx,
                                                               const int32_t *chunk_base,
                                                               const int32_t *offsets,
                                                               int32_t *perm, int32_t *inv,
                                                               int *status) {
    extern __shared__ int s_next[];  // 8 warps x E
    int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int c = blockIdx.x * 8 + wid;
    int nchunks = (T + CH - 1) / CH;
    if (c >= nchunks) return;
    int *nx = s_next + wid * E;
    for (int e = lane; e < E; e += 32) nx[e] = offsets[e] + chunk_base[(int64_t)c * E + e];
    __syncwarp();
    int64_t f0 = (int64_t)c * CH * k;
    int64_t f1 = min((int64_t)(c + 1) * CH, (int64_t)T) * k;
    warp_stable_scatter(idx, f0, f1, E, nx, perm, inv, status);
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
    return moe_launch_plan_build(T, E, k, p, ws, status, st);
}

cudaError_t moe_launch_plan_build(int T, int E, int k, const moe_plan_buf *p, void *ws, int *status,
                                  cudaStream_t st) {
    int CH = MOE_PLAN_CHUNK;
    int nchunks = (T + CH - 1) / CH;
    int32_t *chunk = (int32_t *)ws;
    size_t sm = (size_t)8 * E * sizeof(int);
    moe_plan_count_kernel<<<(nchunks + 7) / 8, 256, sm, st>>>(T, E, k, CH, p->topk_idx, chunk,
                                                              status);
    moe_plan_scan_kernel<<<1, 1024, 0, st>>>(T, E, k, nchunks, chunk, p->counts, p->offsets,
                                             p->active);
    moe_plan_scatter_kernel<<<(nchunks + 7) / 8, 256, sm, st>>>(T, E, k, CH, p->topk_idx, chunk,
                                                                p->offsets, p->perm, p->inv,
                                                                status);
    return cudaGetLastError();
}
