// Device code shared by the routing kernels: keys and top-k of a warp, scans
// and the single-CTA plan.
#pragma once

#include "common.cuh"
#include "kernels.h"

#define FULL_MASK 0xFFFFFFFFu

namespace moe_route {

// Order-preserving 32-bit key of a logit: a larger key is a larger value;
// -0 and +0 share a key (they compare equal). NaN is mapped to -inf first.
__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

// Keys of one warp's k largest: lane l holds key[i] of position l + 32 i
// (i < NK); positions order equal keys. Returns in lane j < k the j-th
// selection's position and key (descending key, ties to the lower
// position). `scratch` is k entries of warp-private shared memory.
//
// Selection by threshold rather than k rounds of arg-max: a bitwise search
// finds the k-th largest key t (the largest x with at least k keys >= x),
// stopping early once exactly k keys are >= the prefix found so far; every
// key > t is selected, and of the keys equal to t the lowest positions fill
// the remaining places. The k winners are then ranked by (key, position).
// The per-lane counts are summed in independent partial sums: a single
// dependent chain over a lane's keys made each of the 32 steps several
// hundred cycles.
template <int NK>
__device__ __forceinline__ void warp_select(const uint32_t (&key)[NK], int k, int lane,
                                            uint2 *scratch, int &pos_out, uint32_t &key_out) {
    uint32_t thr = 0u;
    for (int b = 31; b >= 0; --b) {
        const uint32_t cand = thr | (1u << b);
        int c[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NK; ++i) c[i & 3] += key[i] >= cand ? 1 : 0;
        const int tot =
            (int)__reduce_add_sync(FULL_MASK, (unsigned)((c[0] + c[1]) + (c[2] + c[3])));
        if (tot >= k) {
            thr = cand;
            if (tot == k) break;  // the keys >= thr are the selection
        }
    }
    uint32_t sel = 0u;
    int gt = 0;
#pragma unroll
    for (int i = 0; i < NK; ++i)
        if (key[i] > thr) {
            sel |= 1u << i;
            ++gt;
        }
    int need = k - (int)__reduce_add_sync(FULL_MASK, (unsigned)gt);  // keys equal to thr to take
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        if (need > 0) {  // warp-uniform
            // row i holds positions 32 i + lane: lower lane = lower position
            const uint32_t m = __ballot_sync(FULL_MASK, key[i] == thr);
            const int take = min(need, __popc(m));
            if (((m >> lane) & 1u) && __popc(m & lanemask_lt()) < take) sel |= 1u << i;
            need -= take;
        }
    }
    // compact the k selections into scratch, then rank them
    const int mine = __popc(sel);
    int pos = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(FULL_MASK, pos, off);
        if (lane >= off) pos += o;
    }
    pos -= mine;
#pragma unroll
    for (int i = 0; i < NK; ++i)
        if ((sel >> i) & 1u) scratch[pos++] = make_uint2(key[i], (uint32_t)(lane + 32 * i));
    __syncwarp();
    uint2 me = make_uint2(0u, 0u);
    int r[4] = {0, 0, 0, 0};
    if (lane < k) {
        me = scratch[lane];
#pragma unroll
        for (int q = 0; q < MOE_MAX_TOPK; ++q) {
            if (q < k) {
                const uint2 o = scratch[q];
                r[q & 3] += (o.x > me.x || (o.x == me.x && o.y < me.y)) ? 1 : 0;
            }
        }
    }
    __syncwarp();
    if (lane < k) scratch[(r[0] + r[1]) + (r[2] + r[3])] = me;
    __syncwarp();
    pos_out = -1;
    key_out = 0u;
    if (lane < k) {
        const uint2 w = scratch[lane];
        pos_out = (int)w.y;
        key_out = w.x;
    }
    __syncwarp();
}

// Key of expert e of a logit row (NaN counts as -inf and sets nan_seen);
// positions past E get key 0, below every real key.
__device__ __forceinline__ uint32_t row_key(const float *row, int e, int E, bool &nan_seen) {
    if (e >= E) return 0u;
    float t = row[e];
    if (t != t) {
        nan_seen = true;
        t = -INFINITY;
    }
    return logit_key(t);
}

// Sort value of expert e's logit key: larger is earlier in the selection
// order (descending logit, then ascending index); all values distinct.
__device__ __forceinline__ uint64_t sort_value(uint32_t key, int e) {
    return ((uint64_t)key << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)e);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int m) {
    const uint32_t lo = __shfl_xor_sync(FULL_MASK, (uint32_t)v, m);
    const uint32_t hi = __shfl_xor_sync(FULL_MASK, (uint32_t)(v >> 32), m);
    return ((uint64_t)hi << 32) | lo;
}

// Sorts P independent sets of 64 values in descending order, interleaved so
// that their dependent chains overlap: element n = 2 lane + h of set p in
// v[p][h]. Bitonic network: for block size K = 2 .. 64 and distance
// J = K / 2 .. 1, element n is paired with n ^ J and the pair ordered
// descending where (n & K) == 0, ascending elsewhere (the last block, K = 64,
// orders everything descending).
template <int P>
__device__ __forceinline__ void warp_sort64(uint64_t (&v)[P][2], int lane) {
#pragma unroll
    for (int K = 2; K <= 64; K <<= 1) {
#pragma unroll
        for (int J = K >> 1; J > 0; J >>= 1) {
            if (J == 1) {  // partners in the same lane
                const bool desc = ((2 * lane) & K) == 0;
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const uint64_t a = v[q][0], b = v[q][1];
                    const uint64_t mx = a > b ? a : b, mn = a > b ? b : a;
                    v[q][0] = desc ? mx : mn;
                    v[q][1] = desc ? mn : mx;
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int n = 2 * lane + h;
                    const bool take_max = (((n & K) == 0) == ((n & J) == 0));
#pragma unroll
                    for (int q = 0; q < P; ++q) {
                        const uint64_t o = shfl_xor64(v[q][h], J >> 1);
                        v[q][h] = take_max ? (v[q][h] > o ? v[q][h] : o) : (v[q][h] > o ? o : v[q][h]);
                    }
                }
            }
        }
    }
}

// Top-k of a warp's keys, as warp_select, by a threshold instead of a
// bitwise search when it can: the k-th largest of the 32 lanes' maxima is at
// most the k-th largest key (the k lanes with the largest maxima hold k keys
// at least that large), so every selected key is >= it. When at most 64 keys
// are, they are gathered (with their positions) and sorted by one bitonic
// network, and the first k are the selection. Otherwise (many keys equal or
// close to it) warp_select decides. About 500 instructions per warp against
// the bitwise search's 32 compares per lane and bit, which left a batch of
// one warp per token issue-bound. scratch: 64 x 8 bytes of warp-private
// shared memory (as uint2: 64 entries).
template <int NK>
__device__ __forceinline__ void warp_select_thr(const uint32_t (&key)[NK], int k, int lane,
                                                uint2 *scratch, int &pos_out, uint32_t &key_out) {
    if (k > 16) {  // the k-th largest of 32 maxima bounds too little: nearly always > 64 keys
        warp_select<NK>(key, k, lane, scratch, pos_out, key_out);
        return;
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < NK; ++i) m = key[i] > m ? key[i] : m;
    // the lane maxima in descending order over the lanes (bitonic, as
    // warp_sort64 with one value per lane)
#pragma unroll
    for (int K = 2; K <= 32; K <<= 1) {
#pragma unroll
        for (int J = K >> 1; J > 0; J >>= 1) {
            const uint32_t o = __shfl_xor_sync(FULL_MASK, m, J);
            const bool take_max = ((lane & K) == 0) == ((lane & J) == 0);
            m = take_max ? (m > o ? m : o) : (m > o ? o : m);
        }
    }
    const uint32_t t0 = __shfl_sync(FULL_MASK, m, k - 1);
    int c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < NK; ++i) c[i & 1] += key[i] >= t0 ? 1 : 0;
    const int mine = c[0] + c[1];
    const int total = (int)__reduce_add_sync(FULL_MASK, (unsigned)mine);
    if (total > 64) {
        warp_select<NK>(key, k, lane, scratch, pos_out, key_out);
        return;
    }
    int off = mine;  // exclusive prefix of the lanes' counts
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(FULL_MASK, off, d);
        if (lane >= d) off += o;
    }
    off -= mine;
    uint64_t *cand = reinterpret_cast<uint64_t *>(scratch);
#pragma unroll
    for (int i = 0; i < NK; ++i)
        if (key[i] >= t0) cand[off++] = sort_value(key[i], lane + 32 * i);
    __syncwarp();
    uint64_t v[1][2];
    v[0][0] = 2 * lane < total ? cand[2 * lane] : 0ull;
    v[0][1] = 2 * lane + 1 < total ? cand[2 * lane + 1] : 0ull;
    __syncwarp();
    warp_sort64<1>(v, lane);
    // selection j is element j of the sorted 64: lane j / 2, half j % 2
    const int src = (lane >> 1) & 15;
    const uint32_t lo0 = __shfl_sync(FULL_MASK, (uint32_t)v[0][0], src);
    const uint32_t hi0 = __shfl_sync(FULL_MASK, (uint32_t)(v[0][0] >> 32), src);
    const uint32_t lo1 = __shfl_sync(FULL_MASK, (uint32_t)v[0][1], src);
    const uint32_t hi1 = __shfl_sync(FULL_MASK, (uint32_t)(v[0][1] >> 32), src);
    pos_out = -1;
    key_out = 0u;
    if (lane < k) {
        pos_out = (int)(0xFFFFFFFFu - ((lane & 1) ? lo1 : lo0));
        key_out = (lane & 1) ? hi1 : hi0;
    }
}

// Warp-cooperative top-k of one token's logits (k <= 32, k <= E <= 1024).
// On return lane j < k holds the j-th selection (expert index, logit):
// descending logit, ties to the lower expert index. NaN logits count as -inf
// and set nan_seen. Lane l owns experts l, l + 32, ... (coalesced loads).
// THR: the threshold select (fewer dependent steps: the small-batch plan,
// where one warp's latency is the time); else the bitwise search (fewer
// instructions: the large-batch kernel, where many warps share each SM and
// the threshold select measured 1.8x slower). scratch: 64 entries of
// warp-private shared memory (k entries without THR).
template <bool THR>
__device__ __forceinline__ void warp_topk(const float *row, int E, int k, int lane, int &my_e,
                                          float &my_v, bool &nan_seen, uint2 *scratch) {
    uint32_t key[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) key[i] = row_key(row, lane + 32 * i, E, nan_seen);
    uint32_t kv;
    if constexpr (THR)
        warp_select_thr<32>(key, k, lane, scratch, my_e, kv);
    else
        warp_select<32>(key, k, lane, scratch, my_e, kv);
    my_v = lane < k ? key_logit(kv) : -INFINITY;
}

// Softmax over the k selected logits held by lanes 0..k-1.
__device__ __forceinline__ float warp_select_weight(float my_v, int k, int lane) {
    float vmax = __shfl_sync(FULL_MASK, my_v, 0);
    float ex = (lane < k) ? expf(my_v - vmax) : 0.f;
    float s = ex;
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(FULL_MASK, s, off);
    return ex / s;
}

// Exclusive block scan of one int per thread over a block of NW warps.
template <int NW>
__device__ __forceinline__ int block_exclusive_scan(int v, int *warp_tot, int &total) {
    int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        int o = __shfl_up_sync(FULL_MASK, inc, off);
        if (lane >= off) inc += o;
    }
    if (lane == 31) warp_tot[wid] = inc;
    __syncthreads();
    if (wid == 0) {
        int t = lane < NW ? warp_tot[lane] : 0;
        int ti = t;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            int o = __shfl_up_sync(FULL_MASK, ti, off);
            if (lane >= off) ti += o;
        }
        warp_tot[lane] = ti - t;  // exclusive prefix of warp totals
        if (lane == 31) warp_tot[32] = ti;
    }
    __syncthreads();
    int r = warp_tot[wid] + inc - v;
    total = warp_tot[32];
    __syncthreads();
    return r;
}

// mask[e]: the tokens of chunk c (of MOE_PLAN_CHUNK) that chose expert e, a bit
// each; a token chooses an expert at most once, so a mask holds both the
// expert's rows in the chunk and the order among them. Block-wide.
__device__ __forceinline__ void plan_chunk_mask(uint32_t *mask, int T, int E, int k, int c,
                                                const int32_t *__restrict__ idx, int *status) {
    static_assert(MOE_PLAN_CHUNK == 32, "a bit per token");
    for (int e = threadIdx.x; e < E; e += blockDim.x) mask[e] = 0u;
    __syncthreads();
    const int64_t f0 = (int64_t)c * MOE_PLAN_CHUNK * k;
    const int nf = (int)(min((int64_t)(c + 1) * MOE_PLAN_CHUNK, (int64_t)T) * k - f0);
    for (int i = threadIdx.x; i < nf; i += blockDim.x) {
        const int e = idx[f0 + i];
        if (e >= 0 && e < E) atomicOr(&mask[e], 1u << (i / k));
        else moe_flag(status, MOE_ERR_BAD_INDEX);
    }
    __syncthreads();
}

constexpr int kPlanSmallThreads = 512;
constexpr int kPlanSmallWarps = kPlanSmallThreads / 32;

// Shared memory of the single-CTA plan: T <= 64 tokens, k <= 32. Each expert
// keeps a bit mask of the tokens that chose it. A token chooses an expert at
// most once, so the stable position of flat entry t*k+j (expert e) is
// offsets[e] + the number of tokens before t that chose e.
struct PlanSmall {
    int cnt[MOE_MAX_EXPERTS];
    unsigned long long mask[MOE_MAX_EXPERTS];
    int idx[64 * MOE_MAX_TOPK];
    uint2 scr[kPlanSmallWarps][64];  // each warp's top-k scratch
    int tot[33];
    int nan;
};

__device__ __forceinline__ void plan_small_init(PlanSmall &s) {
    for (int e = threadIdx.x; e < MOE_MAX_EXPERTS; e += kPlanSmallThreads) {
        s.cnt[e] = 0;
        s.mask[e] = 0ull;
    }
    if (threadIdx.x == 0) s.nan = 0;
    __syncthreads();
}

// Lane j < k records token t's j-th selection.
__device__ __forceinline__ void plan_small_put(PlanSmall &s, int t, int k, int lane, int e, float w,
                                               int32_t *topk_idx, float *topk_w) {
    if (lane < k) {
        topk_idx[(int64_t)t * k + lane] = e;
        topk_w[(int64_t)t * k + lane] = w;
        s.idx[t * k + lane] = e;
        atomicAdd(&s.cnt[e], 1);
        atomicOr(&s.mask[e], 1ull << t);
    }
}

// counts, offsets, active, perm and inv from the selections.
__device__ __forceinline__ void plan_small_finish(PlanSmall &s, int T, int E, int k, bool nan_seen,
                                                  const moe_plan_buf &p, int *status) {
    static_assert(2 * kPlanSmallThreads == MOE_MAX_EXPERTS, "two experts per thread in the scans");
    const int tid = threadIdx.x;
    if (__any_sync(FULL_MASK, nan_seen) && (tid & 31) == 0) s.nan = 1;
    __syncthreads();
    if (tid == 0 && s.nan) moe_flag(status, MOE_ERR_NAN_LOGIT);
    // experts e0 = 2 tid and e0 + 1 (counts are zero past E)
    const int e0 = 2 * tid;
    const int c0 = e0 < E ? s.cnt[e0] : 0, c1 = e0 + 1 < E ? s.cnt[e0 + 1] : 0;
    int total;
    const int off = block_exclusive_scan<kPlanSmallWarps>(c0 + c1, s.tot, total);
    const int a0 = c0 > 0 ? 1 : 0, a1 = c1 > 0 ? 1 : 0;
    const int a = block_exclusive_scan<kPlanSmallWarps>(a0 + a1, s.tot, total);
    if (e0 < E) {
        p.counts[e0] = c0;
        p.offsets[e0] = off;
        if (a0) p.active[1 + a] = e0;
    }
    if (e0 + 1 < E) {
        p.counts[e0 + 1] = c1;
        p.offsets[e0 + 1] = off + c0;
        if (a1) p.active[1 + a + a0] = e0 + 1;
    }
    if (tid == 0) {
        p.offsets[E] = T * k;
        p.active[0] = total;
    }
    __syncthreads();
    if (e0 < E) s.cnt[e0] = off;
    if (e0 + 1 < E) s.cnt[e0 + 1] = off + c0;
    __syncthreads();
    for (int f = tid; f < T * k; f += kPlanSmallThreads) {
        const int t = f / k, e = s.idx[f];
        const int pos = s.cnt[e] + __popcll(s.mask[e] & ((1ull << t) - 1ull));
        p.perm[pos] = f;
        p.inv[f] = pos;
    }
}

}  // namespace moe_route
