// Residual addition, RMS norm and E4M3 rows with block scales, in one pass.
//
//   h = bf16(x + r),  y = h / sqrt(mean(h^2) + eps) * w,
//   per 128 columns s = max(max|y| / 448, 2^-126), code = e4m3(y / s)
//
// fp32 throughout. Bound: each of x, r, h, y moves 2 bytes an element, the codes 1.
// A block owns a row and holds it in registers between the sum and the output: a
// thread has chunks of 8 columns, a block's width apart, so that 16 neighbouring
// lanes have a scale's 128 columns.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace {

constexpr int kThreads = 256;

// Two fp32 values to E4M3 (round to nearest even, saturating), the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int CH>
__global__ void __launch_bounds__(kThreads) moe_norm_kernel(MoeNormArgs a) {
    __shared__ float part[kThreads / 32];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, chunks = a.d / 8;
    grid_dep_wait();
    grid_dep_launch();
    float v[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = tid + i * kThreads;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (c >= chunks) continue;
        rope::unpack8(*(const uint4 *)(a.x + t * a.x_stride + 8 * c), v[i]);
        if (a.residual) {
            float r[8];
            rope::unpack8(*(const uint4 *)(a.residual + t * a.residual_stride + 8 * c), r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            const uint4 h = rope::pack8(v[i]);
            if (a.total) *(uint4 *)(a.total + t * a.total_stride + 8 * c) = h;
            rope::unpack8(h, v[i]);  // the norm reads what is stored
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    float inv = 1.f;
    if (a.weight) {
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if ((tid & 31) == 0) part[tid >> 5] = ss;
        __syncthreads();
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) ss += part[i];
        inv = rsqrtf(ss / (float)a.d + a.eps);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = tid + i * kThreads;
        if (a.weight && c < chunks) {
            float w[8];
            rope::unpack8(*(const uint4 *)(a.weight + 8 * c), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * w[j];
        }
        if (a.y && c < chunks) *(uint4 *)(a.y + t * a.y_stride + 8 * c) = rope::pack8(v[i]);
        if (!a.q) continue;
        // the block's largest magnitude by its bits: NaN is above infinity, and both above all else
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (c >= chunks) continue;
        const float s = fmaxf(__uint_as_float(m) / 448.f, 1.17549435e-38f), r = 1.f / s;
        uint32_t q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            q[k] = to_e4m3x2(v[i][4 * k] * r, v[i][4 * k + 1] * r) |
                   to_e4m3x2(v[i][4 * k + 2] * r, v[i][4 * k + 3] * r) << 16;
        *(uint2 *)(a.q + t * a.q_stride + 8 * c) = make_uint2(q[0], q[1]);
        if ((c & 15) == 0)
            a.s[t * a.s_stride + c / 16] = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : s;
    }
}

template <int CH>
cudaError_t launch(const MoeNormArgs &a, cudaStream_t st) {
    return launch_pdl_ready(moe_norm_kernel<CH>, dim3((unsigned)a.T), dim3(kThreads), 0, st, a);
}

}  // namespace

cudaError_t moe_norm_setup() {
    const void *kernels[] = {(const void *)moe_norm_kernel<1>, (const void *)moe_norm_kernel<2>,
                             (const void *)moe_norm_kernel<4>, (const void *)moe_norm_kernel<8>};
    for (const void *k : kernels) {
        const cudaError_t err = set_kernel(k);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

cudaError_t moe_launch_norm(const MoeNormArgs &a, int nsm, cudaStream_t st) {
    const int per = (a.d / 8 + kThreads - 1) / kThreads;
    return per <= 1 ? launch<1>(a, st) : per <= 2 ? launch<2>(a, st) : per <= 4 ? launch<4>(a, st) : launch<8>(a, st);
}
