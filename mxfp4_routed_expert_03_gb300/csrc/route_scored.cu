// Scored routing: scores of the logits (softmax or sigmoid), a balance bias,
// groups of experts, top-k and renormalised weights, then the route plan.
//
// Definition (all fp32): p = softmax(l) or sigmoid(l); s = p + bias; a group's
// score is the sum of its one or two largest s; the best groups are kept, and
// the top-k of s among their experts is the selection, ties to the lower
// index throughout; weights p[e], divided by their sum if asked, times scale.
//
// The selection compares s bit for bit, so it is made from CUDA's expf and
// the correctly rounded fp32 divide, and the softmax's denominator is the sum
// of the exponentials rounded once: a warp adds them as unevaluated pairs of
// floats (Knuth's two-sum), whose total is exact to about 2^-45, in any order.
//
// Bound: 4 E bytes per token from HBM; the instructions of the selection come
// close to it. Without groups every score is first taken approximately (two
// MUFU operations instead of expf and a divide); the k-th largest of the 32
// lanes' maxima is a lower bound of the k-th score, what lies above it (less
// the approximation's error, twice) is a candidate, and only the candidates,
// about one per lane, get their exact score and are ranked (16384 tokens of 896
// experts: 38 us, 56 with exact scores throughout; softmax 45 and 76). More than
// 64 candidates (many equal scores, k near 32) and groups take exact scores of
// all experts.
#include "route.cuh"

using namespace moe_route;

namespace {

// The largest k that is selected among candidates: 16384 tokens of 896 experts
// take 44 us so with k = 20 and 58 with 24 (93 and 94 with a search over the bits
// of all keys), but 108 (96) with 32, where few rows have at most 64 candidates.
constexpr int kMaxCandidateK = 24;

struct ScoreArgs {
    int E, k;
    moe_route_desc r;
    const float *bias;
};

// s + c <- a + (s + c) with the rounding error of the sum kept in c.
__device__ __forceinline__ void two_add(float &s, float &c, float a) {
    const float t = __fadd_rn(s, a);
    const float b = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(a, b)));
    s = t;
}

// exp(l - max), 1 where l is the maximum (infinite ones too).
__device__ __forceinline__ float soft_exp(float l, float mx) {
    return l == mx ? 1.f : expf(__fsub_rn(l, mx));
}

// Score of a logit (not NaN); mx and sum are the softmax's.
template <bool SIGMOID>
__device__ __forceinline__ float score_of(float l, float mx, float sum) {
    if constexpr (SIGMOID) return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-l)));
    return __fdiv_rn(soft_exp(l, mx), sum);
}

__device__ __forceinline__ float load_logit(const float *row, int e, bool &nan_seen) {
    const float l = row[e];
    if (l != l) {
        nan_seen = true;
        return -INFINITY;
    }
    return l;
}

// The two largest keys of the lanes with `in` set.
__device__ __forceinline__ void warp_top2(uint32_t key, bool in, int lane, uint32_t &t1, uint32_t &t2) {
    const uint32_t v = in ? key : 0u;
    t1 = __reduce_max_sync(FULL_MASK, v);
    const int first = __ffs(__ballot_sync(FULL_MASK, v == t1)) - 1;
    t2 = __reduce_max_sync(FULL_MASK, lane == first ? 0u : v);
}

// Keeps in key[] only the experts of the best groups (the others become 0,
// below every real key). A group's score comes from its largest keys, found
// with warp-wide maxima; lane g then ranks group g.
template <int NK>
__device__ __forceinline__ void keep_groups(uint32_t (&key)[NK], const ScoreArgs &a, int lane) {
    const int gs = a.E / a.r.n_groups;
    uint32_t b1 = 0u, b2 = 0u;  // lane g: group g's two largest keys
    auto add = [&](int g, uint32_t t1, uint32_t t2) {
        if (lane == g) {
            b2 = max(max(b2, min(b1, t1)), t2);
            b1 = max(b1, t1);
        }
    };
    if (gs >= 32) {  // a row (experts 32 i ..) lies in one group or two
        int g = 0, end = gs;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            if (32 * i < a.E) {
                uint32_t t1, t2;
                if (end >= 32 * i + 32) {
                    warp_top2(key[i], true, lane, t1, t2);
                    add(g, t1, t2);
                } else {
                    warp_top2(key[i], 32 * i + lane < end, lane, t1, t2);
                    add(g, t1, t2);
                    warp_top2(key[i], 32 * i + lane >= end, lane, t1, t2);
                    add(g + 1, t1, t2);
                }
                if (end <= 32 * i + 32) ++g, end += gs;
            }
        }
    } else {
        for (int g = 0; g < a.r.n_groups; ++g) {
            uint32_t m1 = 0u, m2 = 0u, t2;
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const int e = lane + 32 * i;
                const uint32_t v = (e >= g * gs && e < (g + 1) * gs) ? key[i] : 0u;
                m2 = max(m2, min(m1, v));
                m1 = max(m1, v);
            }
            const uint32_t t1 = __reduce_max_sync(FULL_MASK, m1);
            const int first = __ffs(__ballot_sync(FULL_MASK, m1 == t1)) - 1;
            t2 = __reduce_max_sync(FULL_MASK, lane == first ? m2 : m1);
            add(g, t1, t2);
        }
    }
    const uint32_t mine = lane >= a.r.n_groups ? 0u
                          : a.r.group_top == 1 ? b1
                                               : logit_key(__fadd_rn(key_logit(b1), key_logit(b2)));
    int better = 0;
    for (int g = 0; g < a.r.n_groups; ++g) {
        const uint32_t o = __shfl_sync(FULL_MASK, mine, g);
        better += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    const uint32_t kept =
        __ballot_sync(FULL_MASK, lane < a.r.n_groups && better < a.r.topk_groups);
    // group of expert lane + 32 i, without a division per slot
    int g = lane / gs, rem = lane % gs;
    const int dg = 32 / gs, dr = 32 % gs;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        if (!((kept >> g) & 1u)) key[i] = 0u;  // (past E the key is 0 already)
        g += dg;
        rem += dr;
        if (rem >= gs) rem -= gs, ++g;
        g = min(g, 31);
    }
}

// The sort key of an exact score.
__device__ __forceinline__ uint32_t select_key(float p, float bias, bool &nan_seen) {
    p = __fadd_rn(p, bias);
    if (!(p < INFINITY)) {  // NaN, or an infinite bias
        nan_seen = true;
        p = -INFINITY;
    }
    return logit_key(p);
}

// Values of lanes in descending order over the lanes (bitonic).
__device__ __forceinline__ uint32_t warp_sort32(uint32_t m, int lane) {
#pragma unroll
    for (int K = 2; K <= 32; K <<= 1) {
#pragma unroll
        for (int J = K >> 1; J > 0; J >>= 1) {
            const uint32_t o = __shfl_xor_sync(FULL_MASK, m, J);
            const bool take_max = ((lane & K) == 0) == ((lane & J) == 0);
            m = take_max ? (m > o ? m : o) : (m > o ? o : m);
        }
    }
    return m;
}

// Positions of a warp's candidates: bit i of `mine` is expert lane + 32 i. Writes
// the experts of up to 64 to scratch[].y and returns how many there are.
__device__ __forceinline__ int gather_candidates(uint32_t mine, int lane, uint2 *scratch) {
    const int c = __popc(mine);
    int at = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(FULL_MASK, at, d);
        if (lane >= d) at += o;
    }
    const int n = __shfl_sync(FULL_MASK, at, 31);
    at -= c;
    if (n <= 64)
        for (; mine; mine &= mine - 1u) scratch[at++].y = (uint32_t)(lane + 32 * (__ffs(mine) - 1));
    __syncwarp();
    return n;
}

// The k first of n <= 64 candidates (key, expert) in scratch: lane j < k gets
// the j-th expert.
__device__ __forceinline__ int rank_candidates(uint2 *scratch, int n, int k, int lane) {
    const uint2 c0 = lane < n ? scratch[lane] : make_uint2(0u, 0u);
    int r0 = 0;
#pragma unroll 4
    for (int q = 0; q < n; ++q) {
        const uint2 o = scratch[q];
        r0 += o.x > c0.x || (o.x == c0.x && o.y < c0.y) ? 1 : 0;
    }
    uint2 c1 = make_uint2(0u, 0u);
    int r1 = k;
    if (n > 32) {
        if (lane + 32 < n) c1 = scratch[lane + 32], r1 = 0;
        for (int q = 0; q < n; ++q) {
            const uint2 o = scratch[q];
            r1 += o.x > c1.x || (o.x == c1.x && o.y < c1.y) ? 1 : 0;
        }
    }
    __syncwarp();
    if (lane < n && r0 < k) scratch[r0] = c0;
    if (r1 < k) scratch[r1] = c1;
    __syncwarp();
    const int e = lane < k ? (int)scratch[lane].y : -1;
    __syncwarp();
    return e;
}

template <int NK>
__device__ __forceinline__ void load_row(const float *row, int E, int lane, float (&v)[NK]) {
#pragma unroll
    for (int i = 0; i < NK; ++i) v[i] = lane + 32 * i < E ? row[lane + 32 * i] : -INFINITY;
}

// The biases, 0 without, -inf past E, up to 32 NK. Block-wide, not synchronised.
template <int NK>
__device__ __forceinline__ void load_bias(const ScoreArgs &a, float *bias) {
    for (int e = threadIdx.x; e < 32 * NK; e += blockDim.x)
        bias[e] = e >= a.E ? -INFINITY : a.bias ? a.bias[e] : 0.f;
}

// Softmax of the lane's logits in place: v becomes the exponentials. Returns
// their sum, rounded once; mx: the largest logit. Each lane sums from 1, which
// no exponential exceeds: the rounding error of a sum is then three operations;
// the 32 ones go at the end.
template <int NK>
__device__ __forceinline__ float warp_exps(float (&v)[NK], float &mx) {
    mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NK; ++i) mx = fmaxf(mx, v[i]);
#pragma unroll
    for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, off));
    float s = 1.f, c = 0.f;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        v[i] = soft_exp(v[i], mx);
        const float t = __fadd_rn(s, v[i]);
        c = __fadd_rn(c, __fsub_rn(v[i], __fsub_rn(t, s)));
        s = t;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        const float so = __shfl_xor_sync(FULL_MASK, s, off);
        c = __fadd_rn(c, __shfl_xor_sync(FULL_MASK, c, off));
        two_add(s, c, so);
    }
    return __fadd_rn(__fsub_rn(s, 32.f), c);  // (the difference is exact)
}

// Selection from approximate scores, -1 in all lanes where it does not apply.
// v: the logits, or for the softmax the exponentials; overwritten. The approximation's
// error is below 2^-21 (sigmoid) or 2^-22 of the largest score (softmax), and
// an addition's rounding; the bound takes off four times that, twice.
template <int NK, bool SIGMOID>
__device__ __forceinline__ int warp_select_approx(const float *row, float (&v)[NK], const float *bias,
                                                  const ScoreArgs &a, float mx, float sum, int lane,
                                                  uint2 *scratch) {
    const float L2E = 1.44269504088896341f;
    const float inv = SIGMOID ? 1.f : __frcp_rn(sum);
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        float p;
        if constexpr (SIGMOID) {
            float x;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(v[i] * -L2E));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(1.f + x));
        } else {
            p = v[i] * inv;
        }
        v[i] = p + bias[lane + 32 * i];
        best = fmaxf(best, v[i]);  // (leaves NaN out)
    }
    const float t = key_logit(__shfl_sync(FULL_MASK, warp_sort32(logit_key(best), lane), a.k - 1));
    if (!(fabsf(t) < INFINITY)) return -1;  // warp-uniform
    const float bound = t - (SIGMOID ? 0x1p-18f : 0x1p-19f) * (inv + fabsf(t));
    uint32_t mine = 0u;
#pragma unroll
    for (int i = 0; i < NK; ++i)
        if (!(v[i] < bound)) mine |= 1u << i;  // (NaN too, so that it is seen below)
    const int n = gather_candidates(mine, lane, scratch);
    if (n > 64) return -1;
    bool bad = false;  // an expert that counts as -inf is no candidate
    for (int j = lane; j < n; j += 32) {
        const int e = (int)scratch[j].y;
        const float p = score_of<SIGMOID>(load_logit(row, e, bad), mx, sum);
        scratch[j].x = select_key(p, bias[e], bad);
    }
    __syncwarp();
    if (__any_sync(FULL_MASK, bad)) return -1;
    return rank_candidates(scratch, n, a.k, lane);
}

// One warp's token: lane j < k gets the j-th selected expert and its weight.
// v: the token's logits (-inf past E), overwritten. scratch: 64 entries of
// warp-private shared memory.
template <int NK, bool SIGMOID>
__device__ __forceinline__ void warp_scored_topk(const float *row, float (&v)[NK], const float *bias,
                                                 const ScoreArgs &a, int lane, int &my_e, float &my_w,
                                                 bool &nan_seen, uint2 *scratch) {
    float mx = 0.f, sum = 1.f;
    if constexpr (!SIGMOID) sum = warp_exps<NK>(v, mx);
    my_e = -1;
    // (a row without a finite logit or with a NaN takes the other way)
    const bool plain = a.r.n_groups == 1 && a.k <= kMaxCandidateK &&
                       (SIGMOID || (fabsf(mx) < INFINITY && sum > 0.f));
    if (plain) my_e = warp_select_approx<NK, SIGMOID>(row, v, bias, a, mx, sum, lane, scratch);
    if (!plain || !__any_sync(FULL_MASK, my_e >= 0)) {
        load_row(row, a.E, lane, v);
#pragma unroll
        for (int i = 0; i < NK; ++i)
            if (v[i] != v[i]) {
                nan_seen = true;
                v[i] = -INFINITY;
            }
        if constexpr (!SIGMOID) {
            sum = warp_exps<NK>(v, mx);
            if (mx == -INFINITY) sum = (float)a.E;  // (slots past E count 1 too, then)
        }
        uint32_t key[NK], best = 0u;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            key[i] = 0u;
            if (lane + 32 * i < a.E)
                key[i] = select_key(SIGMOID ? score_of<true>(v[i], 0.f, 1.f) : __fdiv_rn(v[i], sum),
                                    bias[lane + 32 * i],
                                    nan_seen);
        }
        if (a.r.n_groups > 1) keep_groups<NK>(key, a, lane);
        int n = 65;
        if (a.k <= kMaxCandidateK) {  // as above, with exact keys
#pragma unroll
            for (int i = 0; i < NK; ++i) best = max(best, key[i]);
            const uint32_t t = __shfl_sync(FULL_MASK, warp_sort32(best, lane), a.k - 1);
            uint32_t mine = 0u;
#pragma unroll
            for (int i = 0; i < NK; ++i)
                if (key[i] >= t && key[i] > 0u) mine |= 1u << i;
            n = gather_candidates(mine, lane, scratch);
            if (n <= 64) {
                const int c = __popc(mine);
                int at = c;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(FULL_MASK, at, d);
                    if (lane >= d) at += o;
                }
                at -= c;
#pragma unroll
                for (int i = 0; i < NK; ++i)
                    if ((mine >> i) & 1u) scratch[at++].x = key[i];
                __syncwarp();
                my_e = rank_candidates(scratch, n, a.k, lane);
            }
        }
        if (n > 64) {
            uint32_t kv;
            warp_select<NK>(key, a.k, lane, scratch, my_e, kv);
        }
    }
    float w = 0.f;
    if (lane < a.k) {
        bool ignored = false;
        w = score_of<SIGMOID>(load_logit(row, my_e, ignored), mx, sum);
    }
    if (a.r.renormalise) {
        float t = w;
#pragma unroll
        for (int off = 16; off; off >>= 1) t += __shfl_xor_sync(FULL_MASK, t, off);
        w = t > 0.f ? w / t : 0.f;
    }
    my_w = w * a.r.scale;
}

// Small batches: as moe_plan_small_kernel, one CTA, a warp per token.
template <int NK, bool SIGMOID>
__global__ void __launch_bounds__(kPlanSmallThreads) moe_plan_scored_small_kernel(
    int T, ScoreArgs a, const float *__restrict__ logits, moe_plan_buf p, int *status) {
    __shared__ PlanSmall s;
    __shared__ float s_bias[32 * NK];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    load_bias<NK>(a, s_bias);
    plan_small_init(s);
    bool nan_seen = false;
    float v[NK];
    for (int t = wid; t < T; t += kPlanSmallWarps) {
        int my_e;
        float my_w;
        load_row(logits + (int64_t)t * a.E, a.E, lane, v);
        warp_scored_topk<NK, SIGMOID>(logits + (int64_t)t * a.E, v, s_bias, a, lane, my_e, my_w, nan_seen,
                                      s.scr[wid]);
        plan_small_put(s, t, a.k, lane, my_e, my_w, p.topk_idx, p.topk_w);
    }
    plan_small_finish(s, T, a.E, a.k, nan_seen, p, status);
}

// Large batches: a block per chunk of 32 tokens, and the chunk's rows per expert.
// Threads of a block: a warp per token while every SM has one block at most,
// else half as many, two blocks an SM, so that one's start and end overlap the
// other's work (us with 1024 and with 512 threads: 4099 tokens of 256 experts 15
// and 18, 4096 of 1000 16 and 21; 16384 of 256 25 and 23, 16384 of 896 41 and 38).
constexpr int kManyThreads = 32 * MOE_PLAN_CHUNK, kFewThreads = kManyThreads / 2;

template <int NK, bool SIGMOID, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) moe_topk_scored_kernel(int T, ScoreArgs a,
                                                              const float *__restrict__ logits,
                                                              int32_t *topk_idx, float *topk_w,
                                                              int32_t *chunk_counts, int *status) {
    constexpr int kWarps = THREADS / 32;
    __shared__ uint2 s_scratch[kWarps][64];
    __shared__ uint32_t s_mask[MOE_MAX_EXPERTS];
    __shared__ float s_bias[32 * NK];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    for (int e = threadIdx.x; e < a.E; e += THREADS) s_mask[e] = 0u;
    load_bias<NK>(a, s_bias);
    __syncthreads();
    bool nan_seen = false;
    float v[NK];
    for (int i = wid; i < MOE_PLAN_CHUNK; i += kWarps) {
        const int t = blockIdx.x * MOE_PLAN_CHUNK + i;
        if (t >= T) break;
        int my_e;
        float my_w;
        load_row(logits + (int64_t)t * a.E, a.E, lane, v);
        warp_scored_topk<NK, SIGMOID>(logits + (int64_t)t * a.E, v, s_bias, a, lane, my_e, my_w, nan_seen,
                                      s_scratch[wid]);
        if (lane < a.k) {
            topk_idx[(int64_t)t * a.k + lane] = my_e;
            topk_w[(int64_t)t * a.k + lane] = my_w;
            atomicOr(&s_mask[my_e], 1u << i);
        }
    }
    if (__any_sync(FULL_MASK, nan_seen) && lane == 0) moe_flag(status, MOE_ERR_NAN_LOGIT);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += THREADS)
        chunk_counts[(int64_t)blockIdx.x * a.E + e] = __popc(s_mask[e]);
}

template <int NK, bool SIGMOID>
cudaError_t launch(int T, const ScoreArgs &a, const float *logits, const moe_plan_buf *p, void *ws,
                   int *status, int nsm, cudaStream_t st) {
    if (moe_plan_is_small(T))
        return launch_pdl_ready(moe_plan_scored_small_kernel<NK, SIGMOID>, dim3(1),
                          dim3(kPlanSmallThreads), 0, st, T, a, logits, *p, status);
    const int nchunks = (T + MOE_PLAN_CHUNK - 1) / MOE_PLAN_CHUNK;
    const cudaError_t err =
        nchunks <= nsm
            ? launch_pdl_ready(moe_topk_scored_kernel<NK, SIGMOID, kManyThreads>, dim3(nchunks), dim3(kManyThreads), 0,
                               st, T, a, logits, p->topk_idx, p->topk_w, (int32_t *)ws, status)
            : launch_pdl_ready(moe_topk_scored_kernel<NK, SIGMOID, kFewThreads>, dim3(nchunks), dim3(kFewThreads), 0,
                               st, T, a, logits, p->topk_idx, p->topk_w, (int32_t *)ws, status);
    return err != cudaSuccess ? err : moe_launch_plan_build(T, a.E, a.k, true, p, ws, status, st);
}

template <int NK>
cudaError_t setup() {
    const void *kernels[] = {(const void *)moe_plan_scored_small_kernel<NK, true>,
                             (const void *)moe_plan_scored_small_kernel<NK, false>,
                             (const void *)moe_topk_scored_kernel<NK, true, kManyThreads>,
                             (const void *)moe_topk_scored_kernel<NK, false, kManyThreads>,
                             (const void *)moe_topk_scored_kernel<NK, true, kFewThreads>,
                             (const void *)moe_topk_scored_kernel<NK, false, kFewThreads>};
    for (const void *k : kernels) {
        const cudaError_t err = set_kernel(k);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t moe_plan_scored_setup() {
    cudaError_t err = setup<8>();
    if (err == cudaSuccess) err = setup<28>();
    return err != cudaSuccess ? err : setup<32>();
}

cudaError_t moe_launch_plan_scored(int T, int E, int k, const float *logits,
                                   const moe_route_desc &r, const float *bias,
                                   const moe_plan_buf *p, void *ws, int *status, int nsm, cudaStream_t st) {
    const ScoreArgs a = {E, k, r, bias};
    // Slots of a lane: 8, 28 or 32, three kinds of six kernels each. What lies between pays
    // for empty slots: 16384 tokens of 384 experts 31 us (sigmoid) and 40 (softmax), with 16
    // slots 26 and 31; of 512 experts 32 and 26.
    const bool sig = r.score == MOE_SCORE_SIGMOID;
    if (E <= 256)
        return sig ? launch<8, true>(T, a, logits, p, ws, status, nsm, st)
                   : launch<8, false>(T, a, logits, p, ws, status, nsm, st);
    if (E <= 896)
        return sig ? launch<28, true>(T, a, logits, p, ws, status, nsm, st)
                   : launch<28, false>(T, a, logits, p, ws, status, nsm, st);
    return sig ? launch<32, true>(T, a, logits, p, ws, status, nsm, st)
               : launch<32, false>(T, a, logits, p, ws, status, nsm, st);
}
