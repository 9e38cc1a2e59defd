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
// Bound: 4 E bytes per token from HBM; one warp per token keeps the E <= 1024
// sort keys in registers (32 per lane).
#include "route.cuh"

using namespace moe_route;

namespace {

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

// Keeps in key[] only the experts of the best groups (the others become 0,
// below every real key). A group's score comes from its largest keys, found
// with warp-wide maxima; lane g then ranks group g.
template <int NK>
__device__ __forceinline__ void keep_groups(uint32_t (&key)[NK], const ScoreArgs &a, int lane) {
    const int gs = a.E / a.r.n_groups;
    uint32_t mine = 0u;  // lane g: group g's score as a key
    for (int g = 0; g < a.r.n_groups; ++g) {
        uint32_t m1 = 0u, m2 = 0u;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int e = lane + 32 * i;
            const uint32_t v = (e >= g * gs && e < (g + 1) * gs) ? key[i] : 0u;
            m2 = max(m2, min(m1, v));
            m1 = max(m1, v);
        }
        const uint32_t t1 = __reduce_max_sync(FULL_MASK, m1);
        uint32_t sk = t1;
        if (a.r.group_top == 2) {
            const int first = __ffs(__ballot_sync(FULL_MASK, m1 == t1)) - 1;
            const uint32_t t2 = __reduce_max_sync(FULL_MASK, lane == first ? m2 : m1);
            const float v = __fadd_rn(key_logit(t1), key_logit(t2));
            sk = logit_key(v);
        }
        if (lane == g) mine = sk;
    }
    int better = 0;
    for (int g = 0; g < a.r.n_groups; ++g) {
        const uint32_t o = __shfl_sync(FULL_MASK, mine, g);
        better += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    const uint32_t kept =
        __ballot_sync(FULL_MASK, lane < a.r.n_groups && better < a.r.topk_groups);
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int e = lane + 32 * i;
        if (e < a.E && !((kept >> (e / gs)) & 1u)) key[i] = 0u;
    }
}

// One warp's token: lane j < k gets the j-th selected expert and its weight.
// scratch as for warp_topk.
template <int NK, bool SIGMOID, bool THR>
__device__ __forceinline__ void warp_scored_topk(const float *row, const ScoreArgs &a, int lane,
                                                 int &my_e, float &my_w, bool &nan_seen,
                                                 uint2 *scratch) {
    uint32_t key[NK];
    float mx = -INFINITY, sum = 1.f;
    float v[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < a.E ? load_logit(row, e, nan_seen) : -INFINITY;
    }
    if constexpr (!SIGMOID) {
#pragma unroll
        for (int i = 0; i < NK; ++i) mx = fmaxf(mx, v[i]);
#pragma unroll
        for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, off));
        float s = 0.f, c = 0.f;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int e = lane + 32 * i;
            v[i] = e < a.E ? soft_exp(v[i], mx) : 0.f;
            two_add(s, c, v[i]);
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            const float so = __shfl_xor_sync(FULL_MASK, s, off);
            c = __fadd_rn(c, __shfl_xor_sync(FULL_MASK, c, off));
            two_add(s, c, so);
        }
        sum = __fadd_rn(s, c);
    }
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0u;
        if (e < a.E) {
            float p = SIGMOID ? score_of<true>(v[i], 0.f, 1.f) : __fdiv_rn(v[i], sum);
            if (a.bias) p = __fadd_rn(p, a.bias[e]);
            if (!(p < INFINITY)) {  // NaN, or an infinite bias
                nan_seen = true;
                p = -INFINITY;
            }
            key[i] = logit_key(p);
        }
    }
    if (a.r.n_groups > 1) keep_groups<NK>(key, a, lane);
    uint32_t kv;
    if constexpr (THR)
        warp_select_thr<NK>(key, a.k, lane, scratch, my_e, kv);
    else
        warp_select<NK>(key, a.k, lane, scratch, my_e, kv);
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
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    plan_small_init(s);
    bool nan_seen = false;
    for (int t = wid; t < T; t += kPlanSmallWarps) {
        int my_e;
        float my_w;
        warp_scored_topk<NK, SIGMOID, true>(logits + (int64_t)t * a.E, a, lane, my_e, my_w,
                                            nan_seen, s.scr[wid]);
        plan_small_put(s, t, a.k, lane, my_e, my_w, p.topk_idx, p.topk_w);
    }
    plan_small_finish(s, T, a.E, a.k, nan_seen, p, status);
}

template <int NK, bool SIGMOID>
__global__ void __launch_bounds__(256) moe_topk_scored_kernel(int T, ScoreArgs a,
                                                              const float *__restrict__ logits,
                                                              int32_t *topk_idx, float *topk_w,
                                                              int *status) {
    __shared__ uint2 s_scratch[8][64];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int t = blockIdx.x * 8 + wid;
    if (t >= T) return;
    int my_e;
    float my_w;
    bool nan_seen = false;
    warp_scored_topk<NK, SIGMOID, false>(logits + (int64_t)t * a.E, a, lane, my_e, my_w, nan_seen,
                                         s_scratch[wid]);
    if (lane < a.k) {
        topk_idx[(int64_t)t * a.k + lane] = my_e;
        topk_w[(int64_t)t * a.k + lane] = my_w;
    }
    if (__any_sync(FULL_MASK, nan_seen) && lane == 0) moe_flag(status, MOE_ERR_NAN_LOGIT);
}

template <int NK, bool SIGMOID>
cudaError_t launch(int T, const ScoreArgs &a, const float *logits, const moe_plan_buf *p, void *ws,
                   int *status, cudaStream_t st) {
    if (moe_plan_is_small(T))
        return launch_pdl(moe_plan_scored_small_kernel<NK, SIGMOID>, dim3(1),
                          dim3(kPlanSmallThreads), 0, st, T, a, logits, *p, status);
    moe_topk_scored_kernel<NK, SIGMOID><<<(T + 7) / 8, 256, 0, st>>>(T, a, logits, p->topk_idx,
                                                                    p->topk_w, status);
    return moe_launch_plan_build(T, a.E, a.k, p, ws, status, st);
}

}  // namespace

cudaError_t moe_launch_plan_scored(int T, int E, int k, const float *logits,
                                   const moe_route_desc &r, const float *bias,
                                   const moe_plan_buf *p, void *ws, int *status, cudaStream_t st) {
    const ScoreArgs a = {E, k, r, bias};
    const bool sig = r.score == MOE_SCORE_SIGMOID;
    if (E <= 256)
        return sig ? launch<8, true>(T, a, logits, p, ws, status, st)
                   : launch<8, false>(T, a, logits, p, ws, status, st);
    return sig ? launch<32, true>(T, a, logits, p, ws, status, st)
               : launch<32, false>(T, a, logits, p, ws, status, st);
}
