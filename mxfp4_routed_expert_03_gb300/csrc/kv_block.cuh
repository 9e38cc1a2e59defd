// One MXFP4 block of the key/value cache: where it lies and how it is written.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace kv {

// Eight fp32 values to E2M1 codes, the first in the lowest nibble (round to
// nearest even, saturating).
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Slot of a token, split into page-head base and offset; false: skip it.
__device__ __forceinline__ bool slot_ok(const MoeKvArgs &a, int slot) {
    if (slot >= 0 && slot < a.n_slots) return true;
    if (slot != -1) moe_flag(a.status, MOE_ERR_BAD_INDEX);
    return false;
}

// Byte offset of block 0 of a token's codes (blocks 128 bytes apart).
template <int NB>
__device__ __forceinline__ int64_t code_offset(const MoeKvArgs &a, int slot, int head) {
    const int page = slot >> a.page_shift, o = slot & ((1 << a.page_shift) - 1);
    const int64_t ph = (int64_t)page * a.n_kv + head;
    return ((ph << a.page_shift) * NB + (int64_t)(o >> 3) * 8 * NB + (o & 7)) * 16;
}

// Offset of the scale byte of block b: [token][block] for the keys,
// [token pair][block][2] for the values.
template <int NB>
__device__ __forceinline__ int64_t scale_offset(const MoeKvArgs &a, int slot, int head, int b,
                                                bool is_v) {
    const int page = slot >> a.page_shift, o = slot & ((1 << a.page_shift) - 1);
    const int64_t tok = (((int64_t)page * a.n_kv + head) << a.page_shift) + o;
    return is_v ? ((tok >> 1) * NB + b) * 2 + (o & 1) : tok * NB + b;
}

// Writes block b of a token's head: 32 bf16 values in w.
template <int NB>
__device__ __forceinline__ void write_block(const MoeKvArgs &a, bool is_v, int slot, int head, int b,
                                            const uint32_t (&w)[16]) {
    // the largest magnitude as bf16 bits (ordered as integers, NaN highest)
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    // scale byte: exponent field - 2, at least 0 (2^-127); its inverse is 2^(127 - byte)
    const uint32_t byte = (uint32_t)max((int)(m >> 7) - 2, 0);
    const float inv = __uint_as_float((254u - byte) << 23);
    uint32_t code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[4 * i + j] << 16) * inv;
            v[2 * j + 1] = __uint_as_float(w[4 * i + j] & 0xFFFF0000u) * inv;
        }
        code[i] = to_e2m1x8(v);
    }
    *(uint4 *)((is_v ? a.c.v_q : a.c.k_q) + code_offset<NB>(a, slot, head) + 128 * b) =
        make_uint4(code[0], code[1], code[2], code[3]);
    (is_v ? a.c.v_s : a.c.k_s)[scale_offset<NB>(a, slot, head, b, is_v)] =
        (uint8_t)(m >= 0x7F80u ? 255u : byte);
}

}  // namespace kv
