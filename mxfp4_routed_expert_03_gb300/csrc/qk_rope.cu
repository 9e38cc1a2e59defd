// Per-head RMS norm and position rotation of queries and keys, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then for the first rope_dim elements
//   (a, b) -> (a cos - b sin, b cos + a sin),
//
// fp32 throughout, rounded once to bf16. Bound: 2 bytes read and 2 written per
// element. D / 16 threads own a head row and each holds two 16-byte chunks of
// it, chosen so that a rotated pair always lies in one thread: chunks i and
// i + rope_dim/16 of the rotated part (halves apart, a pair is element j of
// both; interleaved, a pair lies inside a chunk), the unrotated rest in
// neighbouring pairs. A warp keeps one token, so the cosines and sines stay in
// registers over its heads.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void unpack8(const uint4 &u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp takes P passes of 32 / (D / 16) head rows of one token; rows [0, n_q)
// are the queries', the next n_k the keys'. `groups` warps share a token.
template <int D, int P>
__global__ void __launch_bounds__(32 * kWarps) moe_qk_norm_rope_kernel(MoeRopeArgs a, int T, int groups) {
    constexpr int TPH = D / 16;   // threads per head row
    constexpr int HP = 32 / TPH;  // head rows per warp and pass
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const uint32_t task = blockIdx.x * kWarps + wid, token = task / groups, group = task - token * groups;
    const int64_t t = token;
    const int i = lane % TPH, rows = a.n_q + a.n_k;
    const int row0 = group * P * HP + lane / TPH;
    grid_dep_wait();
    grid_dep_launch();
    if (token >= (uint32_t)T) return;
    const int np = a.rope_dim / 16;
    const bool turn = i < np;
    const int c0 = turn ? i : 2 * np + 2 * (i - np), c1 = turn ? i + np : c0 + 1;
    const int pos = np > 0 ? a.positions[t] : 0;  // (in flight beside the rows)
    uint4 raw[P][2];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int r = row0 + p * HP;
        raw[p][0] = raw[p][1] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
            const uint16_t *src = r < a.n_q ? a.q + t * a.q_stride + (int64_t)r * D
                                            : a.k + t * a.k_stride + (int64_t)(r - a.n_q) * D;
            raw[p][0] = *(const uint4 *)(src + 8 * c0);
            raw[p][1] = *(const uint4 *)(src + 8 * c1);
        }
    }
    if (np > 0) {
        if (pos < 0 || pos >= a.n_pos) {
            if (lane == 0 && group == 0) moe_flag(a.status, MOE_ERR_BAD_INDEX);
            return;
        }
    }
    // halves: cs[j] / sn[j] belong to pair j of the thread (element j of both
    // chunks); interleaved: pairs 0..3 lie in the first chunk, 4..7 in the second
    float cs[8], sn[8];
    if (turn) {
        const float *tab = a.cos_sin + (int64_t)pos * a.rope_dim;
        const int o0 = a.interleaved ? 4 * c0 : 8 * i, o1 = a.interleaved ? 4 * c1 : 8 * i + 4;
        const float4 x0 = *(const float4 *)(tab + o0), x1 = *(const float4 *)(tab + o1);
        tab += a.rope_dim / 2;
        const float4 y0 = *(const float4 *)(tab + o0), y1 = *(const float4 *)(tab + o1);
        cs[0] = x0.x, cs[1] = x0.y, cs[2] = x0.z, cs[3] = x0.w;
        cs[4] = x1.x, cs[5] = x1.y, cs[6] = x1.z, cs[7] = x1.w;
        sn[0] = y0.x, sn[1] = y0.y, sn[2] = y0.z, sn[3] = y0.w;
        sn[4] = y1.x, sn[5] = y1.y, sn[6] = y1.z, sn[7] = y1.w;
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int r = row0 + p * HP;
        const bool is_q = r < a.n_q;
        float x[8], y[8];
        unpack8(raw[p][0], x);
        unpack8(raw[p][1], y);
        const uint16_t *w = is_q ? a.q_weight : a.k_weight;
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
        for (int off = TPH / 2; off; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
        if (r >= rows) continue;
        if (w) {
            const float inv = rsqrtf(ss * (1.f / D) + a.eps);
            float g0[8], g1[8];
            unpack8(*(const uint4 *)(w + 8 * c0), g0);
            unpack8(*(const uint4 *)(w + 8 * c1), g1);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = x[j] * inv * g0[j];
                y[j] = y[j] * inv * g1[j];
            }
        }
        if (turn && !a.interleaved) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = x[j], v = y[j];
                x[j] = u * cs[j] - v * sn[j];
                y[j] = v * cs[j] + u * sn[j];
            }
        } else if (turn) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = x[2 * j], v = x[2 * j + 1], m = y[2 * j], n = y[2 * j + 1];
                x[2 * j] = u * cs[j] - v * sn[j];
                x[2 * j + 1] = v * cs[j] + u * sn[j];
                y[2 * j] = m * cs[4 + j] - n * sn[4 + j];
                y[2 * j + 1] = n * cs[4 + j] + m * sn[4 + j];
            }
        }
        uint16_t *dst = is_q ? a.q_out + t * a.q_out_stride + (int64_t)r * D
                             : a.k_out + t * a.k_out_stride + (int64_t)(r - a.n_q) * D;
        *(uint4 *)(dst + 8 * c0) = pack8(x);
        *(uint4 *)(dst + 8 * c1) = pack8(y);
    }
}

template <int D, int P>
cudaError_t launch(int T, const MoeRopeArgs &a, cudaStream_t st) {
    const int per_warp = P * (32 / (D / 16)), groups = (a.n_q + a.n_k + per_warp - 1) / per_warp;
    const int64_t tasks = (int64_t)T * groups;
    return launch_pdl_ready(moe_qk_norm_rope_kernel<D, P>, dim3((unsigned)((tasks + kWarps - 1) / kWarps)),
                            dim3(32 * kWarps), 0, st, a, T, groups);
}

template <int D>
cudaError_t launch(int T, const MoeRopeArgs &a, int nsm, cudaStream_t st) {
    const int passes = (a.n_q + a.n_k + 32 / (D / 16) - 1) / (32 / (D / 16));
    // few tokens: one pass per warp, so that the rows spread over the SMs (tokens of 64
    // heads, one pass and more: 5 1.9 and 2.7 us, 76 2.1 and 2.9, 152 2.5 and 3.0, 300 3.3
    // and 3.3, 600 5.0 and 5.2, 2000 12.3 and 10.7; the rule changes at 152); else
    // the largest of 4, 3 and 2 that wastes the fewest passes (more loads in
    // flight: 8191 tokens of 72 heads 73 us with 4 passes a warp of which a
    // quarter were empty, 56 us with 3)
    if ((int64_t)T * (a.n_q + a.n_k) < (int64_t)nsm * 64) return launch<D, 1>(T, a, st);
    int best = 4, waste = (passes + 3) / 4 * 4 - passes;
    for (int p = 3; p >= 2; --p) {
        const int w = (passes + p - 1) / p * p - passes;
        if (w < waste) best = p, waste = w;
    }
    return best == 4 ? launch<D, 4>(T, a, st) : best == 3 ? launch<D, 3>(T, a, st) : launch<D, 2>(T, a, st);
}

}  // namespace

cudaError_t moe_qk_norm_rope_setup() {
    const void *kernels[] = {
        (const void *)moe_qk_norm_rope_kernel<64, 1>,  (const void *)moe_qk_norm_rope_kernel<64, 2>,
        (const void *)moe_qk_norm_rope_kernel<64, 3>,  (const void *)moe_qk_norm_rope_kernel<64, 4>,
        (const void *)moe_qk_norm_rope_kernel<128, 1>, (const void *)moe_qk_norm_rope_kernel<128, 2>,
        (const void *)moe_qk_norm_rope_kernel<128, 3>, (const void *)moe_qk_norm_rope_kernel<128, 4>};
    for (const void *k : kernels) {
        const cudaError_t err = set_kernel(k);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

cudaError_t moe_launch_qk_norm_rope(int T, int head_dim, const MoeRopeArgs &a, int nsm,
                                    cudaStream_t st) {
    return head_dim == 64 ? launch<64>(T, a, nsm, st) : launch<128>(T, a, nsm, st);
}
