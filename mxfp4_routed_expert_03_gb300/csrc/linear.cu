// E4M3 rows times an E4M3 weight matrix, both with block scales, on tcgen05
// tensor cores:
//
//   out[t][n] = sum_b x_s[t][b] w_s[n/128][b] sum_{k in block b} x_q[t][k] w_q[n][k]
//
// The scales are any fp32 values, so they cannot go into the tensor core's own
// sums: the products of one 128-wide K block are summed in TMEM (four MMAs; a
// product of two E4M3 codes is exact in fp32) and added, times the block's two
// scales, to fp32 sums in registers, which also rounds to nearest where the
// tensor core's accumulator truncates.
//
// Tiles of 128 rows of x (TMEM lanes, so that a thread has one row and one scale
// factor per block) x 256 weight rows. One persistent CTA per SM, 11 warps: TMA
// producer (one thread), TMEM allocator, MMA issuer (one thread), 8 warps that add
// blocks (two per lane quadrant, 128 columns each); one ring of stages,
// double-buffered TMEM accumulators, every wait bounded. Rows and columns beyond
// the matrices read as zeros and are not stored.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace {

constexpr int BK = 128;  // codes per 128-byte row, a scale block's width
constexpr int BM = 128, BN = 256;
constexpr int kThreads = 352;
constexpr int kStages = 4;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
constexpr int BAR_BASE = kStages * STAGE;
constexpr int SMEM = 1024 + BAR_BASE + 256;
static_assert(STAGE % 1024 == 0 && SMEM <= 232448, "shared memory");

// kind::f8f6f4 instruction descriptor: fp32 accumulator (bit 4), E4M3 A and B
// (both fields 0), both K-major, N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ __forceinline__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] x B[smem]^T, E4M3 operands, 32 K per instruction.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    moe_linear_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX,
                      const MoeLinearArgs args) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *full = (uint64_t *)(smem + BAR_BASE);
    uint64_t *empty = full + kStages;
    uint64_t *cfull = empty + kStages;  // accumulator c % 2 holds block c
    uint64_t *cempty = cfull + 2;
    uint64_t *drain = cempty + 2;  // the issuer's MMAs in flight, waited on when giving up
    uint64_t *never = drain + 1;   // test hook: nothing arrives here
    uint32_t *tmem_slot = (uint32_t *)(never + 1);
    int *abort_flag = (int *)(tmem_slot + 1);
    int *s_issued = abort_flag + 1;  // stages the producer filled
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        *abort_flag = 0;
        *s_issued = 0;
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&cfull[b], 1);
            tc::mbar_init(&cempty[b], 8);
        }
        tc::mbar_init(drain, 1);
        tc::mbar_init(never, 1);
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int MT = (args.T + BM - 1) / BM, NT = (args.N + BN - 1) / BN, KB = (args.K + BK - 1) / BK;
    const int total = MT * NT;
    const long long LIMIT = args.timeout_cycles;
    volatile int *abort_p = abort_flag;
    auto fail = [&](void) {
        *abort_p = 1;
        moe_flag(args.status, MOE_ERR_DEVICE_TIMEOUT);
    };
    grid_dep_wait();
    grid_dep_launch();
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = tc::policy_evict_last();
            int it = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
                const int mt = tile % MT, nt = tile / MT;
                for (int kb = 0; kb < KB; ++kb) {
                    const int s = it % kStages, round = it / kStages;
                    if (round > 0 && !tc::mbar_wait(&empty[s], (round - 1) & 1, LIMIT, abort_p)) {
                        fail();
                        ok = false;
                        break;
                    }
                    unsigned char *st = smem + s * STAGE;
                    tc::mbar_arrive_expect_tx(&full[s], (uint32_t)STAGE);
                    ++it;  // a fill of this stage is now in flight
                    tc::tma_load_2d(st, &mX, &full[s], kb * BK, mt * BM, pol);
                    tc::tma_load_2d(st + A_BYTES, &mW, &full[s], kb * BK, nt * BN, pol);
                    tc::tma_load_2d(st + A_BYTES + B_BYTES / 2, &mW, &full[s], kb * BK, nt * BN + 128, pol);
                }
            }
            *s_issued = it;
        }
    } else if (warp == 2) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            uint64_t *last = nullptr;
            uint32_t last_par = 0;
            for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % kStages, round = it / kStages;
                    const int cb = it & 1, use = it >> 1;
                    if (!tc::mbar_wait(&full[s], round & 1, LIMIT, abort_p) ||
                        (use > 0 && !tc::mbar_wait(&cempty[cb], (use - 1) & 1, LIMIT, abort_p)) ||
                        (args.inject == MOE_INJECT_LINEAR_STALL && it == 1 &&
                         !tc::mbar_wait(never, 0, LIMIT, abort_p))) {
                        fail();
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint32_t a_s = tc::smem_u32(smem + s * STAGE), b_s = a_s + A_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        mma_e4m3(tmem + cb * BN, tc::sdesc_sw128(a_s + 32 * k), tc::sdesc_sw128(b_s + 32 * k),
                                 idesc_e4m3(BM, BN), k > 0 ? 1u : 0u);
                    tc::mma_commit(&empty[s]);
                    tc::mma_commit(&cfull[cb]);
                    last = &cfull[cb];
                    last_par = use & 1;
                }
            }
            // the last MMAs must finish before the CTA releases TMEM
            if (ok && last && !tc::mbar_wait(last, last_par, LIMIT, abort_p)) fail();
            if (!ok || *abort_p) tc::drain_mmas(drain, LIMIT);
        }
        __syncwarp();
    } else if (warp >= 3) {
        const int q = warp & 3;              // TMEM lane quadrant this warp may access
        const int half = (warp - 3) >> 2;    // which 128 weight rows (one scale block)
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + half * 128;
        int it = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
            const int mt = tile % MT, nt = tile / MT;
            const int64_t t = (int64_t)mt * BM + q * 32 + lane;
            const int n0 = nt * BN + half * 128;
            const bool live = t < args.T && n0 < args.N;
            const float *xs = args.x_s + (live ? t * args.x_s_stride : 0);
            const float *ws = args.w_s + (live ? (int64_t)(n0 / 128) * KB : 0);
            float sum[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) sum[j] = 0.f;
            for (int kb = 0; kb < KB; ++kb, ++it) {
                const int cb = it & 1, use = it >> 1;
                const float f = xs[kb] * ws[kb];
                if (!__all_sync(0xFFFFFFFFu, tc::mbar_wait(&cfull[cb], use & 1, LIMIT, abort_p))) {
                    if (lane == 0) fail();
                    ok = false;
                    break;
                }
                tc::tc_fence_after();
#pragma unroll
                for (int b = 0; b < 128; b += 16) {
                    uint32_t r[16];
                    tc::tmem_ld_32x32b_x16(acc + cb * BN + b, r);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[b + j] = fmaf(__uint_as_float(r[j]), f, sum[b + j]);
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&cempty[cb]);
            }
            if (!ok) break;
            if (!live) continue;
            if (args.out_f32) {
                float *o = (float *)args.out + t * args.out_stride + n0;
#pragma unroll
                for (int j = 0; j < 128; j += 4)
                    if (n0 + j < args.N) *(float4 *)(o + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
            } else {
                uint16_t *o = (uint16_t *)args.out + t * args.out_stride + n0;
#pragma unroll
                for (int j = 0; j < 128; j += 8)
                    if (n0 + j < args.N)
                        *(uint4 *)(o + j) = make_uint4(bf16x2(sum[j], sum[j + 1]), bf16x2(sum[j + 2], sum[j + 3]),
                                                       bf16x2(sum[j + 4], sum[j + 5]), bf16x2(sum[j + 6], sum[j + 7]));
            }
        }
    }
    __syncthreads();
    if (*abort_p && tid == 0) tc::wait_issued_fills(full, kStages, *s_issued, LIMIT);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

cudaError_t moe_linear_setup() { return set_kernel((const void *)moe_linear_kernel, SMEM); }

int moe_linear_box_rows(int T, int K, int N, int nsm) { return BM; }

cudaError_t moe_launch_linear(const CUtensorMap &map_w, const CUtensorMap &map_x,
                              const MoeLinearArgs &a, int nsm, cudaStream_t st) {
    const int64_t tiles = (int64_t)((a.T + BM - 1) / BM) * ((a.N + BN - 1) / BN);
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl_ready(moe_linear_kernel, dim3((unsigned)(tiles < nsm ? tiles : nsm)), dim3(kThreads), SMEM, st,
                            map_w, map_x, a);
}
