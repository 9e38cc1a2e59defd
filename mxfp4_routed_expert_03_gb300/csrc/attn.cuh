// Device code shared by the attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace moe_attention {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kTile = 32;  // tokens per tile of the split kernel

// The four bytes of w (two codes each, low nibble first) as four f16 pairs.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// s += a, with c the part by which s is too large (Kahan's summation).
__device__ __forceinline__ void add_to(float &s, float &c, float a) {
    const float y = __fsub_rn(a, c), t = __fadd_rn(s, y);
    c = __fsub_rn(__fsub_rn(t, s), y);
    s = t;
}
__device__ __forceinline__ float pow2(int e) {  // 2^e for e in [-127, 127]
    return __uint_as_float(e == -127 ? 0x00400000u : (uint32_t)(e + 127) << 23);
}


// A sequence as scheduled: its rows, and its items (column tile x head) of
// `tiles` token tiles each, the first at token lo (a multiple of the tile).
struct Seq {
    int q0, nq, kv, lo, tiles, ncol, cts;
};

template <int NC>
__device__ __forceinline__ Seq seq_of(const MoeAttnArgs &a, int b) {
    Seq s;
    const moe_attn_batch &B = a.b;
    int q1 = b + 1;
    s.q0 = b;
    if (B.cu_q) {
        s.q0 = B.cu_q[b];
        q1 = B.cu_q[b + 1];
    }
    s.nq = q1 - s.q0;
    if (s.q0 < 0 || q1 < s.q0 || q1 > B.n_tokens) {
        moe_flag(a.status, MOE_ERR_BAD_INDEX);
        s.q0 = s.nq = 0;
    }
    if (s.nq > B.max_q) {
        moe_flag(a.status, MOE_ERR_BAD_INDEX);
        s.nq = B.max_q;
    }
    s.kv = B.kv_len[b];
    if (s.kv < 0 || s.kv > B.max_kv) {
        moe_flag(a.status, MOE_ERR_BAD_INDEX);
        s.kv = s.kv < 0 ? 0 : B.max_kv;
    }
    s.ncol = s.nq * a.group;
    s.cts = (s.ncol + NC - 1) / NC;
    int lo = 0;
    if (B.window > 0) lo = max(0, s.kv - s.nq + 1 - B.window);
    s.lo = lo / kTile * kTile;
    // at least one tile: rows that see nothing are written too
    s.tiles = max(1, (s.kv - s.lo + kTile - 1) / kTile);
    return s;
}

// Output of elements d, d + 1 of one row and head: o / l, or 0 where no key was seen. `up` is
// what m is less than the maximum that l is taken against.
__device__ __forceinline__ void store_out(const MoeAttnArgs &a, int row, int head, int D, int d,
                                          float o0, float o1, float m, float l, int up) {
    const float r = l == 0.f ? 0.f : 1.f / l;
    *(__nv_bfloat162 *)(a.out + (int64_t)row * a.out_stride + head * D + d) =
        __floats2bfloat162_rn(l == 0.f ? 0.f : o0 * r, l == 0.f ? 0.f : o1 * r);
    if (d == 0 && a.lse)
        a.lse[(int64_t)row * a.n_kv * a.group + head] =
            l == 0.f ? -INFINITY : (m + (log2f(l) + up)) * CUDART_LN2_F;
}

}  // namespace moe_attention
