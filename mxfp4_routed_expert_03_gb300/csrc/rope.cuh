// Norm and rotation of one head row held by D / 16 threads, shared by the
// kernels that write the result to memory (qk_rope.cu) and into the cache
// (rope_append.cu), so that both give the same bits.
//
// Each thread holds two 16-byte chunks of the row, chosen so that a rotated pair
// always lies in one thread: chunks i and i + rope_dim/16 of the rotated part
// (halves apart, a pair is element j of both; interleaved, a pair lies inside a
// chunk), the unrotated rest in neighbouring pairs.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace rope {

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

// What thread i of a row holds.
struct Lane {
    int i, c0, c1;  // its index in the row, its two chunks
    bool turn;      // they are rotated
    __device__ __forceinline__ Lane(int i_, int rope_dim) : i(i_) {
        const int np = rope_dim / 16;
        turn = i < np;
        c0 = turn ? i : 2 * np + 2 * (i - np);
        c1 = turn ? i + np : c0 + 1;
    }
};

// cosines and sines of a position for a thread's pairs. Halves: cs[j] / sn[j]
// belong to pair j of the thread (element j of both chunks); interleaved: pairs
// 0..3 lie in the first chunk, 4..7 in the second.
__device__ __forceinline__ void load_angles(const MoeRopeArgs &a, const Lane &l, int pos,
                                            float (&cs)[8], float (&sn)[8]) {
    const float *tab = a.cos_sin + (int64_t)pos * a.rope_dim;
    const int o0 = a.interleaved ? 4 * l.c0 : 8 * l.i, o1 = a.interleaved ? 4 * l.c1 : 8 * l.i + 4;
    const float4 x0 = *(const float4 *)(tab + o0), x1 = *(const float4 *)(tab + o1);
    tab += a.rope_dim / 2;
    const float4 y0 = *(const float4 *)(tab + o0), y1 = *(const float4 *)(tab + o1);
    cs[0] = x0.x, cs[1] = x0.y, cs[2] = x0.z, cs[3] = x0.w;
    cs[4] = x1.x, cs[5] = x1.y, cs[6] = x1.z, cs[7] = x1.w;
    sn[0] = y0.x, sn[1] = y0.y, sn[2] = y0.z, sn[3] = y0.w;
    sn[4] = y1.x, sn[5] = y1.y, sn[6] = y1.z, sn[7] = y1.w;
}

// Sum of squares of the row, in every one of its threads (all lanes of the warp).
template <int D>
__device__ __forceinline__ float row_squares(const float (&x)[8], const float (&y)[8]) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
    for (int off = D / 32; off; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
    return ss;
}

// The thread's two chunks x and y normed (weight w, or NULL) and rotated.
template <int D>
__device__ __forceinline__ void norm_turn(const MoeRopeArgs &a, const Lane &l, const uint16_t *w,
                                          float ss, const float (&cs)[8], const float (&sn)[8],
                                          float (&x)[8], float (&y)[8]) {
    if (w) {
        const float inv = rsqrtf(ss * (1.f / D) + a.eps);
        float g0[8], g1[8];
        unpack8(*(const uint4 *)(w + 8 * l.c0), g0);
        unpack8(*(const uint4 *)(w + 8 * l.c1), g1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = x[j] * inv * g0[j];
            y[j] = y[j] * inv * g1[j];
        }
    }
    if (l.turn && !a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float u = x[j], v = y[j];
            x[j] = u * cs[j] - v * sn[j];
            y[j] = v * cs[j] + u * sn[j];
        }
    } else if (l.turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = x[2 * j], v = x[2 * j + 1], m = y[2 * j], n = y[2 * j + 1];
            x[2 * j] = u * cs[j] - v * sn[j];
            x[2 * j + 1] = v * cs[j] + u * sn[j];
            y[2 * j] = m * cs[4 + j] - n * sn[4 + j];
            y[2 * j + 1] = n * cs[4 + j] + m * sn[4 + j];
        }
    }
}

}  // namespace rope
