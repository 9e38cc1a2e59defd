// Residual addition, RMS norm and E4M3 rows with block scales, in one pass.
//
//   h = bf16(x + r),  y = h / sqrt(mean(h^2) + eps) * w,
//   per 128 columns s = max(max|y| / 448, 2^-126), code = e4m3(y / s)
//
// h exactly rounded, the rest in fp32; y / s is rounded to fp32 and then to a code. With a norm, y / s is
// 448 p / max|p| of the block for p = h w, which 16 bits hold exactly: the row's factor is not in it, and about one
// quotient in 8000 is half-way between two codes. Codes are computed from that form, so these go to the even code
// whatever the roundings of y and s (see row_out).
// Bound: each of x, r, h, y moves 2 bytes an element, the codes 1; beside that the instructions.
// Some warps of a block own a row and hold it in registers between the sum and the
// output: a thread has CH chunks of 8 columns, the row's threads apart, so that 16
// neighbouring lanes have a scale's 128 columns.
// 8191 rows of 7168 with residual and codes: 65 us (6.3 TB/s of the 412 MB that have
// to move); 4099 rows of 8192, codes alone: 17 us (6.0 TB/s).
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace {

// Two fp32 values to E4M3 (round to nearest even, saturating), the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The largest magnitude of three values, NaN if one is.
__device__ __forceinline__ float max_abs(float x, float y, float z) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// 1 / x within 2^-24 of its size (x, 1 / x normal): an approximate reciprocal and one step of Newton's method.
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return fmaf(r, fmaf(-x, r, 1.f), r);
}

// v[j] * w[j], two at a time (each rounded as one product); v[j] * w[j] + u[j].
__device__ __forceinline__ void mul8(float (&r)[8], const float (&v)[8], const float (&w)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2)
        asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\t"
            "mov.b64 {%0, %1}, a;\n\t}"
            : "=f"(r[j]), "=f"(r[j + 1])
            : "f"(v[j]), "f"(v[j + 1]), "f"(w[j]), "f"(w[j + 1]));
}
__device__ __forceinline__ void mul8(float (&r)[8], const float (&v)[8], float w) {
    const float all[8] = {w, w, w, w, w, w, w, w};
    mul8(r, v, all);
}
__device__ __forceinline__ void fma8(float (&r)[8], const float (&v)[8], float w, const float (&u)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2)
        asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %6};\n\t"
            "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
            : "=f"(r[j]), "=f"(r[j + 1])
            : "f"(v[j]), "f"(v[j + 1]), "f"(w), "f"(u[j]), "f"(u[j + 1]));
}

// 448 / m for m in [2^-119, 2^128), too large by 2^-23.5 to 2^-21.5 of it: 7 + 3 ulp, and a rounding.
__device__ __forceinline__ float above_448_over(float m) { return reciprocal(m * 0x1p-6f) * (7.f + 3 * 0x1p-21f); }

// Sums of eight pairs of bf16 values, each rounded once.
__device__ __forceinline__ uint4 add8(const uint4 &x, const uint4 &y) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&u[i]),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&v[i]));
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

constexpr float kLeast = 0x1p-126f;  // the least scale

// What a thread has of its row: chunk i is chunk tid + i * threads.
struct Place {
    int warps, tid, threads, sub, rows;  // warps of a row, this thread in it, the row of the block's `rows`
    __device__ __forceinline__ explicit Place(int warps_) : warps(warps_) {
        const int wid = threadIdx.x >> 5;
        sub = wid / warps;
        threads = 32 * warps;
        tid = (wid - sub * warps) * 32 + (threadIdx.x & 31);
        rows = blockDim.x / threads;
    }
};

// Row t (of which this thread has the chunks with live[i]) from its loaded chunks to its outputs; `inv_d` = 1 / d.
// `part`: a word of shared memory per warp.
template <int CH, bool RES, bool NORM>
__device__ __forceinline__ void row_out(const MoeNormArgs &a, const Place &p, int64_t t, const bool (&live)[CH],
                                        float inv_d, uint4 (&x)[CH], const uint4 (&r)[CH], const uint4 (&w)[CH], float *part) {
    const int lane = threadIdx.x & 31;
    float v[CH][8];
    float ss = 0.f, rest = 1.f;
    uint16_t *total = RES && a.total ? a.total + t * a.total_stride + 8 * p.tid : nullptr;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        if (RES) {
            x[i] = add8(x[i], r[i]);
            if (total && live[i]) *(uint4 *)(total + 8 * i * p.threads) = x[i];
        }
        rope::unpack8(x[i], v[i]);  // (the norm reads what is stored)
        if (NORM) {
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
        }
    }
    if (NORM) {
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if (p.warps > 1) {
            if (lane == 0) part[threadIdx.x >> 5] = ss;
            __syncthreads();
            ss = lane < p.warps ? part[p.sub * p.warps + lane] : 0.f;
#pragma unroll
            for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        }
        // inv = unit * rest, unit a power of two (0, infinity and NaN as they are), so that v becomes
        // h * w exactly, at y's own size, and y = v * rest
        const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
        const uint32_t bits = __float_as_uint(inv);
        const bool split = inv > 0.f && inv < __uint_as_float(0x7F800000u);
        const float unit = split ? __uint_as_float(bits & 0x7F800000u) : inv;
        if (split) rest = __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float u[8];
            rope::unpack8(w[i], u);
            mul8(v[i], v[i], unit);
            mul8(v[i], v[i], u);
        }
    }
    if (a.y) {
        uint16_t *y = a.y + t * a.y_stride + 8 * p.tid;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float u[8];
            mul8(u, v[i], rest);
            if (live[i]) *(uint4 *)(y + 8 * i * p.threads) = rope::pack8(u);
        }
    }
    if (!a.q) return;
    uint8_t *code = a.q + t * a.q_stride + 8 * p.tid;
    float *scale = a.s + t * a.s_stride + p.tid / 16;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        float m = max_abs(max_abs(v[i][0], v[i][1], v[i][2]), max_abs(v[i][3], v[i][4], v[i][5]),
                          max_abs(v[i][6], v[i][7], 0.f));
#pragma unroll
        for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float top, s, u[8];
        if (NORM) {
            // With the factor slightly above 448 / m a quotient that is half-way comes out on it or up to 6 ulp above
            // (the product's own rounding included), and the mask takes that back; no other is within 8 ulp of one
            // (numerator and denominator have 16 bits). Where the scale is the least one, y / s takes no rounding
            // beyond y's. (Dividing y by its rounded scale leaves the side that a half-way quotient falls to to the
            // roundings: 777 rows of 4096 6.5 us, 6.8 this way; 8191 of 7168 65.2 and 65.4.)
            top = m * rest;
            s = fmaxf(top * (1.f / 448.f), kLeast);
            const float f = s > kLeast ? above_448_over(m) : rest * 0x1p126f;
            const uint32_t mask = s > kLeast ? ~7u : ~0u;
            mul8(u, v[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = __uint_as_float(__float_as_uint(u[j]) & mask);
        } else {
            // h / s correctly rounded: a product with the reciprocal, then with what that leaves of the dividend
            // (Markstein 1990; checked for all 8-bit significands)
            top = m;
            s = fmaxf(m * (1.f / 448.f), kLeast);
            // (the negated quotient, whose sign is turned below: so a negative zero stays one)
            const float f = -reciprocal(s);
            float left[8];
            mul8(u, v[i], f);
            fma8(left, u, s, v[i]);
            fma8(u, left, f, u);
        }
        uint32_t q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            q[k] = (to_e4m3x2(u[4 * k], u[4 * k + 1]) | to_e4m3x2(u[4 * k + 2], u[4 * k + 3]) << 16) ^
                   (NORM ? 0u : 0x80808080u);
        if (!live[i]) continue;
        *(uint2 *)(code + 8 * i * p.threads) = make_uint2(q[0], q[1]);
        if ((p.tid & 15) == 0)  // (top is not below infinity: it is that, or NaN)
            scale[i * p.threads / 16] = top < __uint_as_float(0x7F800000u) ? s : __uint_as_float(0x7FC00000u);
    }
}

// Few rows: a block has each of its rows once.
template <int CH, bool RES, bool NORM>
__global__ void __launch_bounds__(1024) moe_norm_kernel(MoeNormArgs a, int warps) {
    __shared__ float part[32];
    const Place p(warps);
    const int64_t t = (int64_t)blockIdx.x * p.rows + p.sub;
    grid_dep_wait();
    grid_dep_launch();
    uint4 x[CH], r[CH], w[CH];
    bool live[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = p.tid + i * p.threads;
        live[i] = t < a.T && c < a.d / 8;
        x[i] = r[i] = w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (!live[i]) continue;
        x[i] = *(const uint4 *)(a.x + t * a.x_stride + 8 * c);
        if (RES) r[i] = *(const uint4 *)(a.residual + t * a.residual_stride + 8 * c);
        if (NORM) w[i] = *(const uint4 *)(a.weight + 8 * c);
    }
    row_out<CH, RES, NORM>(a, p, t, live, 1.f / (float)a.d, x, r, w, part);
}

// Many rows: a block goes through rows with the next one on its way (two of them, or four chunks a thread, so
// that half as many warps fit: slower). A thread copies what it will read itself, so
// nothing has to be waited for but its own copies.
constexpr int CH_STREAM = 2;

template <bool RES, bool NORM>
__global__ void __launch_bounds__(1024) moe_norm_stream_kernel(MoeNormArgs a, int warps) {
    constexpr int CH = CH_STREAM, PER = RES ? 2 : 1;
    extern __shared__ uint4 ring[];  // [2][CH][x, residual][thread]
    __shared__ float part[2][32];
    const Place p(warps);
    const int64_t step = (int64_t)gridDim.x * p.rows;
    const int n = blockDim.x;
    uint4 *mine = ring + threadIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    uint4 w[CH];
    bool live[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = p.tid + i * p.threads;
        live[i] = c < a.d / 8;
        w[i] = NORM && live[i] ? *(const uint4 *)(a.weight + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
        if (live[i]) continue;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int k = 0; k < PER; ++k) mine[((s * CH + i) * PER + k) * n] = make_uint4(0u, 0u, 0u, 0u);
    }
    int64_t t = (int64_t)blockIdx.x * p.rows + p.sub;
    auto fetch = [&](int64_t row, int s) {
        if (row < a.T) {
            const uint16_t *x = a.x + row * a.x_stride + 8 * p.tid;
            const uint16_t *r = RES ? a.residual + row * a.residual_stride + 8 * p.tid : nullptr;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                if (!live[i]) continue;
                cp_async_16(mine + (s * CH + i) * PER * n, x + 8 * i * p.threads);
                if (RES) cp_async_16(mine + ((s * CH + i) * PER + 1) * n, r + 8 * i * p.threads);
            }
        }
        cp_async_commit();
    };
    const float inv_d = 1.f / (float)a.d;
    fetch(t, 0);
    // (all rows of a block in as many turns, so that its threads meet at the sums)
    const int turns = (int)((a.T - (int64_t)blockIdx.x * p.rows + step - 1) / step);
    for (int k = 0; k < turns; ++k, t += step) {
        const int s = k & 1;
        // (the next row ahead of this one's arrival, or behind it: with a residual's four streams of rows the
        // latter keeps the memory busier, 8191 rows of 7168 65 us against 69, without 4099 rows of 8192 18.8 and 17.1)
        if (!RES) fetch(t + step, s ^ 1);
        cp_async_wait<RES ? 0 : 1>();
        uint4 x[CH], r[CH];
        bool here[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            here[i] = live[i] && t < a.T;
            x[i] = mine[(s * CH + i) * PER * n];
            r[i] = RES ? mine[((s * CH + i) * PER + 1) * n] : make_uint4(0u, 0u, 0u, 0u);
        }
        if (RES) fetch(t + step, s ^ 1);
        row_out<CH, RES, NORM>(a, p, t, here, inv_d, x, r, w, part[s]);
    }
}

int warps_of(int d, int ch) { return (d / 8 + 32 * ch - 1) / (32 * ch); }

template <int CH, bool RES, bool NORM>
cudaError_t launch(const MoeNormArgs &a, cudaStream_t st) {
    const int warps = warps_of(a.d, CH), rows = a.T > 1 && warps < 8 ? 8 / warps : 1;
    return launch_pdl_ready(moe_norm_kernel<CH, RES, NORM>, dim3((unsigned)((a.T + rows - 1) / rows)),
                            dim3(32 * warps * rows), 0, st, a, warps);
}

template <bool RES, bool NORM>
cudaError_t launch(const MoeNormArgs &a, int nsm, cudaStream_t st) {
    // few rows: latency counts (16 rows of 7168 2.8 and 2.9 us, 300 of 1024 2.0 and 2.5, 1216 of 1024 3.7 and 4.0;
    // the rule changes at 8 K elements an SM; 304 of 7168 5.6 and 5.2)
    if ((int64_t)a.T * a.d <= (int64_t)nsm * 8192)
        return a.d <= 8192 ? launch<1, RES, NORM>(a, st) : launch<2, RES, NORM>(a, st);
    const int warps = warps_of(a.d, CH_STREAM), rows = warps < 8 ? 8 / warps : 1, threads = 32 * warps * rows;
    const int smem = 2 * CH_STREAM * (RES ? 2 : 1) * threads * 16;
    // (the registers of 1024 threads on an SM, and at most 128 KB of rows)
    const int64_t blocks = ((int64_t)a.T + rows - 1) / rows, most = (int64_t)nsm * (1024 / threads);
    return launch_pdl_ready(moe_norm_stream_kernel<RES, NORM>, dim3((unsigned)(blocks < most ? blocks : most)),
                            dim3(threads), smem, st, a, warps);
}

template <bool RES, bool NORM>
cudaError_t setup() {
    cudaError_t err = set_kernel((const void *)moe_norm_kernel<1, RES, NORM>);
    if (err == cudaSuccess) err = set_kernel((const void *)moe_norm_kernel<2, RES, NORM>);
    if (err == cudaSuccess)
        err = set_kernel((const void *)moe_norm_stream_kernel<RES, NORM>, 2 * CH_STREAM * (RES ? 2 : 1) * 1024 * 16);
    return err;
}

}  // namespace

cudaError_t moe_norm_setup() {
    cudaError_t err = setup<false, false>();
    if (err == cudaSuccess) err = setup<false, true>();
    if (err == cudaSuccess) err = setup<true, false>();
    return err == cudaSuccess ? setup<true, true>() : err;
}

cudaError_t moe_launch_norm(const MoeNormArgs &a, int nsm, cudaStream_t st) {
    if (a.residual) return a.weight ? launch<true, true>(a, nsm, st) : launch<true, false>(a, nsm, st);
    return a.weight ? launch<false, true>(a, nsm, st) : launch<false, false>(a, nsm, st);
}
