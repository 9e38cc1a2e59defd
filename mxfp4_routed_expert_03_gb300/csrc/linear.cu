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
// Three kernels:
//   few rows (up to 64; more where the weights are few), where reading the weights is what counts: tiles of 128
//   weight rows (TMEM lanes) x 16, 32 or 64 rows of x;
//   many: tiles of 128 rows of x (TMEM lanes, so that a thread has one row and one factor per block) x 128 weight
//   rows;
//   very many: a pair of CTAs on 256 x 256, which halves what an SM reads per product.
// Where tiles are few, the first two split K over the CTAs of a cluster, so that most SMs read; the parts are
// joined through distributed shared memory in the order of the ranks.
//
// In each, one warp copies (TMA), one thread issues the MMAs, 4 or 8 warps add the blocks; one ring of stages,
// several TMEM accumulators, every wait bounded. Rows and columns beyond the matrices read as zeros and are not
// stored.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace {

constexpr int BK = 128;  // codes per 128-byte row, a scale block's width

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

// The four MMAs of a K block: 128 rows of A and N of B, 128-byte rows (32 bytes on is 2 in a descriptor).
template <int N>
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t a_s, uint32_t b_s) {
    const uint64_t a = tc::sdesc_sw128(a_s), b = tc::sdesc_sw128(b_s);
#pragma unroll
    for (int k = 0; k < BK / 32; ++k) mma_e4m3(d, a + 2 * k, b + 2 * k, idesc_e4m3(128, N), k > 0 ? 1u : 0u);
}

// acc += {a0, a1} * {f0, f1} (a: the bits of fp32 values), two at a time.
__device__ __forceinline__ void fma2(float2 &acc, uint32_t a0, uint32_t a1, float f0, float f1) {
    asm volatile("{\n\t.reg .b64 c, a, f;\n\tmov.b64 c, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\tmov.b64 f, {%4, %5};\n\t"
        "fma.rn.f32x2 c, a, f, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "+f"(acc.x), "+f"(acc.y)
        : "r"(a0), "r"(a1), "f"(f0), "f"(f1));
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Four neighbouring outputs.
__device__ __forceinline__ void store4(const MoeLinearArgs &args, int64_t at, float4 v) {
    if (args.out_f32) *(float4 *)((float *)args.out + at) = v;
    else *(uint2 *)((uint16_t *)args.out + at) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
}

// One output.
__device__ __forceinline__ void store1(const MoeLinearArgs &args, int64_t at, float v) {
    if (args.out_f32) ((float *)args.out)[at] = v;
    else ((uint16_t *)args.out)[at] = f32_to_bf16_bits(v);
}

// A ring position: a stage and the parity of its round.
struct Ring {
    int s = 0;
    uint32_t par = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) s = 0, par ^= 1u;
    }
};

// A CTA's part of a tile, [rows][pitch] fp32 in `stage`, goes to the CTAs of the cluster that join `per` of its
// rows each, rank 0 the first: into their `recv` area [S][per][pitch], counted on their `bar`; its own rows stay.
// By one warp, once every CTA of the cluster has its barriers ready, and also where a wait ran out (whatever
// the part holds then): so the parts that a CTA waits for always come.
__device__ __forceinline__ void send_parts(const float *stage, float *recv, uint64_t *bar, int S, int rank, int rows,
                                           int per, int pitch, int lane) {
    const int to = (rank + lane) % S, n = min(per, rows - to * per);
    if (lane > 0 && lane < S && n > 0)
        tc::bulk_copy_s2peer(tc::peer_addr(recv + rank * per * pitch, to), stage + to * per * pitch, n * pitch * 4,
                             tc::peer_addr(bar, to));
    __syncwarp();
}

// Waits for the parts of this CTA's rows, by a warp, also in a CTA that has given up: a copy still on its way
// when the CTAs leave would read or write what is no longer theirs. A CTA of KB blocks at most sends after as many
// waits as it has blocks and groups of scales, each under `limit`; this limit is longer than all of them.
__device__ __forceinline__ bool wait_parts(uint64_t *bar, int KB, long long limit) {
    if (__all_sync(0xFFFFFFFFu, tc::mbar_try_wait(bar, 0))) return true;
    const long long waits = 2 * KB + 8, most = limit < INT64_MAX / waits ? limit * waits : INT64_MAX, t0 = clock64();
    do {
        if (__all_sync(0xFFFFFFFFu, tc::mbar_try_wait(bar, 0))) return true;
    } while (__all_sync(0xFFFFFFFFu, clock64() - t0 <= most));
    return false;
}

// Test hook: whether this CTA's MMA issuer stalls.
__device__ __forceinline__ bool stalls(int inject, int rank, int S) {
    return inject == MOE_INJECT_LINEAR_STALL || (inject == MOE_INJECT_LINEAR_STALL_FIRST && rank == 0) ||
           (inject == MOE_INJECT_LINEAR_STALL_LAST && rank == S - 1);
}

// Four sums of S parts, this CTA's at `own`, the others' `step` apart at `recv`, in the order of the ranks.
template <int S>
__device__ __forceinline__ float4 join(const float *own, const float *recv, int step, int rank) {
    float4 w[S];
#pragma unroll
    for (int k = 0; k < S; ++k) w[k] = *(const float4 *)(k == rank ? own : recv + k * step);
#pragma unroll
    for (int k = 1; k < S; ++k) w[0].x += w[k].x, w[0].y += w[k].y, w[0].z += w[k].z, w[0].w += w[k].w;
    return w[0];
}
__device__ __forceinline__ float4 join(const float *own, const float *recv, int step, int rank, int S) {
    switch (S) {
        case 2: return join<2>(own, recv, step, rank);
        case 3: return join<3>(own, recv, step, rank);
        case 4: return join<4>(own, recv, step, rank);
        case 5: return join<5>(own, recv, step, rank);
        case 6: return join<6>(own, recv, step, rank);
        case 7: return join<7>(own, recv, step, rank);
        default: return join<8>(own, recv, step, rank);
    }
}

// After a timeout, by all threads: the copies and MMAs in flight end before the CTA leaves. A stage's last
// round completes once the adding warps (one thread of each, `adds`) have made up for the accumulators that
// they did not come to read; earlier rounds are complete, since a stage is filled again only behind its MMAs.
template <int STAGES>
__device__ __forceinline__ void wind_down(uint64_t *full, uint64_t *drain, bool issues, bool adds, int drained,
                                          int issued, long long limit) {
    if (issues && tc::elect_one()) tc::drain_mmas(drain, limit);
    if (adds)
        for (int i = max(drained + STAGES, issued - STAGES); i < issued; ++i) tc::mbar_arrive(&full[i % STAGES]);
    __syncthreads();
    if (threadIdx.x == 0) tc::wait_issued_fills(full, STAGES, issued, limit);
}

// ---------------------------------------------------------------------------
// Many rows of x.
// ---------------------------------------------------------------------------

struct Wide {
    static constexpr int THREADS = 384;
    static constexpr int BN = 128;                      // weight rows per tile
    static constexpr int COLS = BN / 2;                 // columns of a warp that adds blocks
    static constexpr int STAGE_BYTES = (128 + BN) * BK;
    static constexpr int STAGES = 4;                    // and TMEM accumulators
    static constexpr int G = 8;                         // blocks whose scales are fetched at a time
    static constexpr int SROW = 132;                    // row of a scale group: 128 rows of x and a gap (banks)
    static constexpr int SC_BASE = STAGES * STAGE_BYTES;  // scales of x [2][G][SROW], of the weights [2][G][2]
    static constexpr int PITCH = BN + 4;                // row of a part (banks)
    static constexpr int RECV = SC_BASE + 2 * G * SROW * 4 + 2 * G * 2 * 4;  // parts [split][rows / split][PITCH]
    static constexpr int BAR = RECV + (128 + 7) * PITCH * 4;
    static constexpr int BYTES = 1024 + BAR + 256;
    static_assert((2 * STAGES + 7) * 8 + 12 <= 256, "barrier area");
    static_assert(STAGE_BYTES % 1024 == 0 && BYTES <= 232448, "shared memory");
    static_assert(128 * PITCH * 4 <= SC_BASE && RECV % 16 == 0, "a part fits over the ring");
    static_assert(8 * 32 * 144 <= 128 * PITCH * 4, "output rows over the parts");
};

// The scales of 8 blocks of K, from block g of nkb on (kb0: the CTA's first), by one warp: of 128 rows of x,
// 8 neighbouring blocks of 4 rows per load, to xsc [block][SROW], and of NB tiles of 128 weight rows to
// wsc [block][2]. `ready` is called between the loads and the stores.
template <int NB, int SROW, typename Ready>
__device__ __forceinline__ bool load_scales(const MoeLinearArgs &args, float *xsc, float *wsc, int t0, int nb, int kb0,
                                            int g, int nkb, int KB, int lane, Ready ready) {
    const int kb = g + (lane & 7), wkb = g + (lane >> 1), wb = nb + (lane & 1);
    float *dst = xsc + (lane & 7) * SROW + (lane >> 3);
    float w = 0.f;
    if (lane < 16 && wkb < nkb && (lane & 1) < NB && wb * 128 < args.N) w = args.w_s[(int64_t)wb * KB + kb0 + wkb];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t t = t0 + 64 * h + 4 * i + (lane >> 3);
            v[i] = kb < nkb && t < args.T ? args.x_s[t * args.x_s_stride + kb0 + kb] : 0.f;
        }
        if (h == 0 && !ready()) return false;
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[64 * h + 4 * i] = v[i];
    }
    if (lane < 16) wsc[lane] = w;
    __syncwarp();
    return true;
}

// A warp's sums over nkb blocks of 32 rows x 2 N2 columns: sum += accumulator * scale, block by block. TMEM is
// read 64 columns ahead of the additions, the next block's barrier is tested and its scale read ahead of
// their use (all of these in turn: 8191 rows of 7168 x 9216 467 us, where that build took 367; 32 columns ahead: 434).
//   acc()           the current block's columns in TMEM
//   wait(), test()  waits for the current block's MMAs, false: given up; whether they are finished
//   drained()       its accumulator has been read: on to the next block
//   scale(kb, f)    block kb's factors of the thread's row and of the columns; false: given up
template <int N2, typename Acc, typename Test, typename Wait, typename Drained, typename Scale>
__device__ __forceinline__ bool add_blocks(float2 (&sum)[N2], int nkb, Acc acc, Test test, Wait wait, Drained drained,
                                           Scale scale) {
    constexpr int P = N2 / 16;  // pieces of 32 columns, in pairs
    uint32_t r[2][32];
    float2 f, next;
    if (!scale(0, f) || !wait()) return false;
    tc::tc_fence_after();
    tc::tmem_ld_32x32b_x32(acc(), r[0]);
    tc::tmem_ld_32x32b_x32(acc() + 32, r[1]);
    for (int kb = 0; kb < nkb; ++kb) {
        const bool more = kb + 1 < nkb;
        const float factor = f.x * f.y;
        const auto add = [&](int p) {
#pragma unroll
            for (int j = 0; j < 16; ++j) fma2(sum[16 * p + j], r[p & 1][2 * j], r[p & 1][2 * j + 1], factor, factor);
        };
#pragma unroll
        for (int p = 0; p < P; p += 2) {
            tc::tmem_ld_wait();
            if (p + 2 < P) {
                add(p);
                tc::tmem_ld_32x32b_x32(acc() + 32 * (p + 2), r[0]);
                add(p + 1);
                tc::tmem_ld_32x32b_x32(acc() + 32 * (p + 3), r[1]);
            } else {
                tc::tc_fence_before();
                __syncwarp();
                drained();
                const bool ready = more && test();
                // (here, where the other warp of the scheduler can add: ahead of the block 421 us, behind add(p)
                // 404, behind the next block's first load 438)
                if (more && !scale(kb + 1, next)) return false;
                add(p);
                if (__all_sync(0xFFFFFFFFu, ready)) {
                    tc::tc_fence_after();
                    tc::tmem_ld_32x32b_x32(acc(), r[0]);
                    add(p + 1);
                    tc::tmem_ld_32x32b_x32(acc() + 32, r[1]);
                } else {
                    add(p + 1);
                    if (more) {
                        if (!wait()) return false;
                        tc::tc_fence_after();
                        tc::tmem_ld_32x32b_x32(acc(), r[0]);
                        tc::tmem_ld_32x32b_x32(acc() + 32, r[1]);
                    }
                }
            }
        }
        f = next;
    }
    return true;
}

// 32 rows x 2 N2 columns of the output, from row t0 and column n0 on, of a warp whose lanes have a row each: SEG
// bytes of every row at a time through `stage` (32 rows of SEG + 16 bytes), so that whole sectors are
// written (16 bytes of each lane's own row at a time: 3.6 us between two tiles).
template <int SEG, int N2>
__device__ __forceinline__ void store_rows(const MoeLinearArgs &args, int64_t t0, int n0, const float2 (&sum)[N2],
                                           unsigned char *stage, int lane) {
    constexpr int PITCH = SEG + 16, L = SEG / 16;  // L lanes copy a row's piece
    unsigned char *mine = stage + lane * PITCH;
    const unsigned char *from = stage + lane / L * PITCH + lane % L * 16;
    const int rows = (int)(args.T - t0 < 32 ? args.T - t0 : 32);
    const auto copy = [&](int col, int width, int bytes) {  // the staged piece, columns n0 + col on
        __syncwarp();
        const int n = n0 + col + lane % L * width;
        unsigned char *out = (unsigned char *)args.out + ((t0 + lane / L) * args.out_stride + n) * bytes;
        if (n < args.N)
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (32 / L * i + lane / L < rows)
                    *(uint4 *)(out + 32 / L * i * args.out_stride * bytes) =
                        *(const uint4 *)(from + 32 / L * i * PITCH);
        __syncwarp();
    };
    if (args.out_f32) {
#pragma unroll
        for (int c = 0; c < 8 * N2 / SEG; ++c) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const float2 *v = sum + SEG / 8 * c + 2 * j;
                *(float4 *)(mine + 16 * j) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
            }
            copy(SEG / 4 * c, 4, 4);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 4 * N2 / SEG; ++c) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const float2 *v = sum + SEG / 4 * c + 4 * j;
                *(uint4 *)(mine + 16 * j) = make_uint4(bf16x2(v[0].x, v[0].y), bf16x2(v[1].x, v[1].y),
                                                       bf16x2(v[2].x, v[2].y), bf16x2(v[3].x, v[3].y));
            }
            copy(SEG / 2 * c, 8, 2);
        }
    }
}

}  // namespace

// Barriers of a stage: `full` completes when its copies have come and the accumulator that its block goes to
// has been read (an arrival of every adding warp), so the issuer has one wait per block; `done` when its MMAs
// are finished: its memory is free, its accumulator is full.
// Bound: an SM takes in about 62 bytes a cycle from L2, 276 ns for the 32 KB of a block (MMAs alone 178 ns, all
// together 306). 333 rows of 4096 x 5120 12.2 us, 2049 of 4096 x 1000 to fp32 12.3: 32 of these blocks, then start
// and end.
__global__ void __launch_bounds__(Wide::THREADS, 1)
    moe_linear_wide_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX,
                           const MoeLinearArgs args) {
    using C = Wide;
    constexpr int BN = C::BN;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *xsc = (float *)(smem + C::SC_BASE), *wsc = xsc + 2 * C::G * C::SROW;
    float *parts = (float *)(smem + C::RECV);
    uint64_t *full = (uint64_t *)(smem + C::BAR);
    uint64_t *done = full + C::STAGES;
    uint64_t *sfull = done + C::STAGES;    // scale group g % 2
    uint64_t *sempty = sfull + 2;
    uint64_t *recv = sempty + 2;           // the parts of this CTA's rows
    uint64_t *drain = recv + 1;            // the issuer's MMAs in flight, waited on when giving up
    uint64_t *never = drain + 1;           // test hook: nothing arrives here
    uint32_t *tmem_slot = (uint32_t *)(never + 1);
    int *abort_flag = (int *)(tmem_slot + 1);
    int *s_issued = abort_flag + 1;        // stages the producer filled
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)tc::cluster_rank(), S = (int)tc::cluster_size();
    const int MT = (args.T + 127) / 128, NT = (args.N + BN - 1) / BN, KB = (args.K + BK - 1) / BK;
    const int total = MT * NT, first = blockIdx.x / S, step = gridDim.x / S;
    const int kb0 = KB * rank / S, nkb = KB * (rank + 1) / S - kb0;
    // split: rows of the (one) tile, how many of them a CTA joins, how many this one does
    const int rows = min(128, args.T - first % MT * 128), per = (rows + S - 1) / S, own = min(per, rows - rank * per);
    if (tid == 0) {
        *abort_flag = 0;
        *s_issued = 0;
        for (int s = 0; s < C::STAGES; ++s) {
            tc::mbar_init(&full[s], 1 + 8);
            tc::mbar_init(&done[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&sfull[b], 1);
            tc::mbar_init(&sempty[b], 8);
        }
        tc::mbar_init(recv, 1);
        tc::mbar_init(drain, 1);
        tc::mbar_init(never, 1);
        tc::fence_mbar_init();
        if (S > 1 && own > 0) tc::mbar_arrive_expect_tx(recv, (S - 1) * own * C::PITCH * 4);
        tc::prefetch_map(&mW);
        tc::prefetch_map(&mX);
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (S > 1) tc::cluster_arrive();  // (1: this CTA's barriers are ready)
    const uint32_t tmem = *tmem_slot;
    const long long LIMIT = args.timeout_cycles;
    volatile int *abort_p = abort_flag;
    auto fail = [&](void) {
        *abort_p = 1;
        moe_flag(args.status, MOE_ERR_DEVICE_TIMEOUT);
    };
    bool ok = true;
    int drained = 0;  // blocks that an adding warp has read
    if (warp == 0 && tc::elect_one()) {  // the first stages' weights on their way to L2 while the kernel before ends
        for (int kb = 0; kb < min(C::STAGES, nkb); ++kb) tc::tma_prefetch_2d(&mW, (kb0 + kb) * BK, first / MT * BN);
    }
    __syncwarp();
    grid_dep_wait();  // (every warp: however long the kernel before takes, no wait below runs out meanwhile)
    grid_dep_launch();
    if (warp < 4) {
        if (warp == 0) {
            const uint64_t pol = tc::policy_evict_last();
            int it = 0;
            Ring at;
            for (int tile = first; tile < total && ok; tile += step) {
                const int t0 = tile % MT * 128, n0 = tile / MT * BN;
                for (int kb = kb0; kb < kb0 + nkb; ++kb, ++it, at.next(C::STAGES)) {
                    if (it >= C::STAGES && !tc::mbar_wait_warp(&done[at.s], at.par ^ 1u, LIMIT, abort_p)) {
                        ok = false;
                        break;
                    }
                    if (tc::elect_one()) {
                        unsigned char *st = smem + at.s * C::STAGE_BYTES;
                        tc::mbar_arrive_expect_tx(&full[at.s], (uint32_t)C::STAGE_BYTES);
                        tc::tma_load_2d(st, &mX, &full[at.s], kb * BK, t0, pol);
                        tc::tma_load_2d(st + 128 * BK, &mW, &full[at.s], kb * BK, n0, pol);
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) *s_issued = it;
        } else if (warp == 2) {
            const bool stall = stalls(args.inject, rank, S);
            int it = 0;
            Ring at;
            for (int tile = first; tile < total && ok; tile += step) {
                for (int kb = 0; kb < nkb; ++kb, ++it, at.next(C::STAGES)) {
                    if (!tc::mbar_wait_warp(&full[at.s], at.par, LIMIT, abort_p) ||
                        (stall && !tc::mbar_wait_warp(never, 0, LIMIT, abort_p))) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    if (tc::elect_one()) {
                        const uint32_t a_s = tc::smem_u32(smem) + at.s * C::STAGE_BYTES;
                        mma_block<BN>(tmem + at.s * BN, a_s, a_s + 128 * BK);
                        tc::mma_commit(&done[at.s]);
                    }
                    __syncwarp();
                }
            }
            // (the last MMAs have finished when the adding warps are through with the last block)
        } else if (warp == 3) {
            int it = 0;
            for (int tile = first; tile < total && ok; tile += step)
                for (int g = 0; g < nkb && ok; g += C::G, ++it) {
                    const int b = it & 1, use = it >> 1;
                    ok = load_scales<1, C::SROW>(args, xsc + b * C::G * C::SROW, wsc + b * 2 * C::G, tile % MT * 128,
                                                 tile / MT, kb0, g, nkb, KB, lane, [&] {
                        return use == 0 || tc::mbar_wait_warp(&sempty[b], (use - 1) & 1, LIMIT, abort_p);
                    });
                    if (ok && lane == 0) tc::mbar_arrive(&sfull[b]);
                }
        }
        if (!ok && lane == 0) fail();
        if (S > 1) {
            __syncwarp();
            tc::cluster_wait();  // (1)
        }
    } else {
        const int q = warp & 3;             // TMEM lane quadrant this warp may access
        const int half = (warp - 4) >> 2;   // which columns
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + half * C::COLS;
        const int row = q * 32 + lane;
        if (lane == 0)
            for (int s = 0; s < C::STAGES; ++s) tc::mbar_arrive(&full[s]);  // (empty accumulators)
        int sg = -1;  // scale group
        Ring at;      // of block `drained`
        for (int tile = first; tile < total; tile += step) {
            const int n0 = tile / MT * BN + half * C::COLS;
            float2 sum[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[j] = make_float2(0.f, 0.f);
            ok = add_blocks(
                sum, nkb, [&] { return acc + at.s * BN; }, [&] { return tc::mbar_test_wait(&done[at.s], at.par); },
                [&] { return tc::mbar_wait_warp(&done[at.s], at.par, LIMIT, abort_p); },
                [&] {
                    if (lane == 0) tc::mbar_arrive(&full[at.s]);
                    ++drained;
                    at.next(C::STAGES);
                },
                [&](int kb, float2 &f) {
                    if (kb % C::G == 0) {
                        if (kb > 0 && lane == 0) tc::mbar_arrive(&sempty[sg & 1]);
                        ++sg;
                        if (!tc::mbar_wait_warp(&sfull[sg & 1], (sg >> 1) & 1, LIMIT, abort_p)) return false;
                    }
                    const int at = (sg & 1) * C::G + kb % C::G;
                    f = make_float2(xsc[at * C::SROW + row], wsc[at * 2]);
                    return true;
                });
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sempty[sg & 1]);
            if (!ok) break;
            if (S > 1) {
                // over the ring, all of whose copies and MMAs are done
                float *o = (float *)smem + row * C::PITCH + half * C::COLS;
#pragma unroll
                for (int j = 0; j < C::COLS / 2; j += 2)
                    *(float4 *)(o + 2 * j) = make_float4(sum[j].x, sum[j].y, sum[j + 1].x, sum[j + 1].y);
                break;  // (one tile per cluster)
            }
            store_rows<128>(args, (int64_t)(tile % MT) * 128 + q * 32, n0, sum, smem + C::RECV + (warp - 4) * 4608,
                            lane);
        }
        if (!ok && lane == 0) fail();
        __syncwarp();  // (the barriers below are for whole warps)
        if (S > 1) {
            tc::fence_proxy_async_smem();
            ok = tc::bar_and(1, 256, ok);
            tc::cluster_wait();  // (1)
            if (warp == 4) send_parts((const float *)smem, parts, recv, S, rank, rows, per, C::PITCH, lane);
            if (own > 0 && !wait_parts(recv, KB, LIMIT)) ok = false;
            if (!ok && lane == 0) fail();
            __syncwarp();
        }
    }
    if (S > 1) {
        tc::cluster_arrive();  // (2: this CTA has the parts of its rows)
        if (warp >= 4 && ok) {
            const int n0 = first / MT * BN;
            const int64_t t0 = first % MT * 128 + rank * per;
            for (int u = tid - 128; u < own * (BN / 4); u += 256) {
                const int r = u / (BN / 4), c = u % (BN / 4) * 4;
                if (n0 + c >= args.N) continue;
                store4(args, (t0 + r) * args.out_stride + n0 + c,
                       join((const float *)smem + (rank * per + r) * C::PITCH + c, parts + r * C::PITCH + c,
                            per * C::PITCH, rank, S));
            }
        }
        __syncwarp();
        tc::cluster_wait();  // (2: all parts have arrived, also where a wait ran out: none is on its way to or from here)
    }
    __syncthreads();
    if (*abort_p) wind_down<C::STAGES>(full, drain, warp == 2, warp >= 4 && lane == 0, drained, *s_issued, LIMIT);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Very many rows of x: a pair of CTAs on a tile of 256 x 256.
// ---------------------------------------------------------------------------
namespace {

struct Pair {
    static constexpr int THREADS = 384;
    static constexpr int STAGE_BYTES = 256 * BK;  // of a CTA: 128 rows of x, 64 of each 128 weight rows
    static constexpr int STAGES = 5;
    static constexpr int G = 8;                   // as in Wide
    static constexpr int SROW = 132;
    static constexpr int SC_BASE = STAGES * STAGE_BYTES;
    static constexpr int OUT = SC_BASE + 2 * G * SROW * 4 + 2 * G * 2 * 4;  // output rows of 8 warps
    static constexpr int BAR = OUT + 8 * 32 * 144;
    static constexpr int BYTES = 1024 + BAR + 512;
    // registers a thread at launch and after the split: 4 warps give, 8 take
    static constexpr int REGS = 168, REGS_LOW = 88, REGS_HIGH = 208;
    static_assert(REGS_LOW + 2 * REGS_HIGH <= 3 * REGS, "the split draws on the launch's registers");
    static_assert((4 * STAGES + 8) * 8 + 12 <= 512 && BYTES <= 232448, "barrier area, shared memory");
};

// As mma_block<128>, for 128 rows of A and 64 of B in each CTA of the pair.
__device__ __forceinline__ void mma_block_pair(uint32_t d, uint32_t a_s, uint32_t b_s) {
    const uint64_t a = tc::sdesc_sw128(a_s), b = tc::sdesc_sw128(b_s);
#pragma unroll
    for (int k = 0; k < BK / 32; ++k)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a + 2 * k), "l"(b + 2 * k), "r"(idesc_e4m3(256, 128)), "r"(k > 0 ? 1u : 0u)
            : "memory");
}

}  // namespace

// Each CTA has 128 rows of x and half of the weight rows' codes; the first CTA's issuer drives both tensor
// cores, and both CTAs have all 256 weight rows for their rows of x in TMEM, as two accumulators of 2 x 128
// columns. The two halves are separate MMAs with barriers of their own, so that one half's sums are read and
// freed while the other is computed; 4 warps add a half's blocks.
// Barriers: `come` in each CTA, its copies; `full` in the first CTA, the copies of both and the first half's
// accumulator read by both; `free1` in the first CTA, the second half's accumulator read by both; `done` in
// each CTA, the MMAs of a half.
// Bound: a block takes 375 ns; its copies alone 306, its additions alone 300, its MMAs alone 274. 8191 rows of 7168 x
// 9216 376 to 387 us (2.8 PFLOP/s), 440 when it runs for seconds at the power limit. 60 bytes a thread are spilled; other
// register splits spill more.
__global__ void __launch_bounds__(Pair::THREADS, 1)
    moe_linear_pair_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX,
                           const MoeLinearArgs args) {
    using C = Pair;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *xsc = (float *)(smem + C::SC_BASE), *wsc = xsc + 2 * C::G * C::SROW;
    uint64_t *come = (uint64_t *)(smem + C::BAR);
    uint64_t *full = come + C::STAGES;
    uint64_t *done = full + C::STAGES;     // [half][stage]
    uint64_t *free1 = done + 2 * C::STAGES;
    uint64_t *sfull = free1 + 2, *sempty = sfull + 2;
    uint64_t *drain = sempty + 2, *never = drain + 1;
    uint32_t *tmem_slot = (uint32_t *)(never + 1);
    int *abort_flag = (int *)(tmem_slot + 1);
    int *s_issued = abort_flag + 1;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)tc::cluster_rank();
    if (tid == 0) {
        *abort_flag = 0;
        *s_issued = 0;
        for (int s = 0; s < C::STAGES; ++s) {
            tc::mbar_init(&come[s], 1);
            tc::mbar_init(&full[s], 2 + 8);
            tc::mbar_init(&done[s], 1);
            tc::mbar_init(&done[C::STAGES + s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&free1[b], 8);
            tc::mbar_init(&sfull[b], 1);
            tc::mbar_init(&sempty[b], 8);
        }
        tc::mbar_init(drain, 1);
        tc::mbar_init(never, 1);
        tc::fence_mbar_init();
        tc::prefetch_map(&mW);
        tc::prefetch_map(&mX);
    }
    if (warp == 1) tc::tmem_alloc_pair(tmem_slot, 512);
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_arrive();
    tc::cluster_wait();  // (barriers and tensor memory of both CTAs are ready)
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int MT = (args.T + 255) / 256, NT = (args.N + 255) / 256, KB = (args.K + BK - 1) / BK;
    const int total = MT * NT, first = blockIdx.x / 2, step = gridDim.x / 2;
    const long long LIMIT = args.timeout_cycles;
    volatile int *abort_p = abort_flag;
    auto fail = [&](void) {
        *abort_p = 1;
        moe_flag(args.status, MOE_ERR_DEVICE_TIMEOUT);
    };
    bool ok = true;
    grid_dep_wait();  // (every warp, as above)
    grid_dep_launch();
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_LOW));
        if (warp == 0) {
            const uint64_t pol = tc::policy_evict_last();
            int it = 0;
            Ring at;
            for (int tile = first; tile < total && ok; tile += step) {
                const int t0 = tile % MT * 256 + rank * 128, n0 = tile / MT * 256 + rank * 64;
                for (int kb = 0; kb < KB; ++kb, ++it, at.next(C::STAGES)) {
                    if (it >= C::STAGES && !tc::mbar_wait_warp(&done[C::STAGES + at.s], at.par ^ 1u, LIMIT, abort_p)) {
                        ok = false;
                        break;
                    }
                    if (tc::elect_one()) {
                        unsigned char *st = smem + at.s * C::STAGE_BYTES;
                        tc::mbar_arrive_expect_tx(&come[at.s], (uint32_t)C::STAGE_BYTES);
                        tc::tma_load_2d(st, &mX, &come[at.s], kb * BK, t0, pol);
                        tc::tma_load_2d(st + 128 * BK, &mW, &come[at.s], kb * BK, n0, pol);
                        tc::tma_load_2d(st + 192 * BK, &mW, &come[at.s], kb * BK, n0 + 128, pol);
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) *s_issued = it;
        } else if (warp == 1) {
            // the copies of this CTA have come: tells the first CTA's issuer
            Ring at;
            for (int tile = first; tile < total && ok; tile += step)
                for (int kb = 0; kb < KB; ++kb, at.next(C::STAGES)) {
                    if (!tc::mbar_wait_warp(&come[at.s], at.par, LIMIT, abort_p)) {
                        ok = false;
                        break;
                    }
                    if (tc::elect_one()) tc::peer_arrive(tc::peer_addr(&full[at.s], 0));
                    __syncwarp();
                }
        } else if (warp == 2 && rank == 0) {
            const bool stall = stalls(args.inject, 0, 2);
            int it = 0;
            Ring at;
            for (int tile = first; tile < total && ok; tile += step) {
                for (int kb = 0; kb < KB; ++kb, ++it, at.next(C::STAGES)) {
                    if (!tc::mbar_wait_warp(&full[at.s], at.par, LIMIT, abort_p) ||
                        (stall && !tc::mbar_wait_warp(never, 0, LIMIT, abort_p))) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint32_t a_s = tc::smem_u32(smem) + at.s * C::STAGE_BYTES, d = tmem + (it & 1) * 256;
                    if (tc::elect_one()) {
                        mma_block_pair(d, a_s, a_s + 128 * BK);
                        tc::mma_commit_pair(&done[at.s], 3u);
                    }
                    __syncwarp();
                    if (it >= 2 && !tc::mbar_wait_warp(&free1[it & 1], ((it >> 1) - 1) & 1, LIMIT, abort_p)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    if (tc::elect_one()) {
                        mma_block_pair(d + 128, a_s, a_s + 192 * BK);
                        tc::mma_commit_pair(&done[C::STAGES + at.s], 3u);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 3) {
            int it = 0;
            for (int tile = first; tile < total && ok; tile += step)
                for (int g = 0; g < KB && ok; g += C::G, ++it) {
                    const int b = it & 1, use = it >> 1;
                    ok = load_scales<2, C::SROW>(args, xsc + b * C::G * C::SROW, wsc + b * 2 * C::G,
                                                 tile % MT * 256 + rank * 128, tile / MT * 2, 0, g, KB, KB, lane, [&] {
                        return use == 0 || tc::mbar_wait_warp(&sempty[b], (use - 1) & 1, LIMIT, abort_p);
                    });
                    if (ok && lane == 0) tc::mbar_arrive(&sfull[b]);
                }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_HIGH));
        const int q = warp & 3, half = (warp - 4) >> 2, col = half * 128;  // TMEM lane quadrant; columns
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + col;
        const int row = q * 32 + lane;
        uint64_t *mine = done + half * C::STAGES;
        // where it tells that accumulator `i & 1` has been read: with the stage that uses it next, or by its number
        const uint32_t told = tc::peer_addr(half ? free1 : full, 0);
        // (only for blocks that come, so that the issuer waits for every arrival: one in flight behind the last
        // wait could reach a CTA that has left)
        const int blocks = (total - first + step - 1) / step * KB;
        if (half == 0 && lane == 0) {
            tc::peer_arrive(told);
            if (blocks > 1) tc::peer_arrive(told + 8);
        }
        int sg = -1, i = 0;  // scale group, block
        Ring at, ahead;      // of block i, of block i + 2
        ahead.s = 2;
        for (int tile = first; tile < total; tile += step) {
            float2 sum[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) sum[j] = make_float2(0.f, 0.f);
            ok = add_blocks(
                sum, KB, [&] { return acc + (i & 1) * 256; }, [&] { return tc::mbar_test_wait(&mine[at.s], at.par); },
                [&] { return tc::mbar_wait_warp(&mine[at.s], at.par, LIMIT, abort_p); },
                [&] {
                    if (lane == 0 && i + 2 < blocks) tc::peer_arrive(told + 8 * (half ? i & 1 : ahead.s));
                    ++i;
                    at.next(C::STAGES);
                    ahead.next(C::STAGES);
                },
                [&](int kb, float2 &f) {
                    if (kb % C::G == 0) {
                        if (kb > 0 && lane == 0) tc::mbar_arrive(&sempty[sg & 1]);
                        ++sg;
                        if (!tc::mbar_wait_warp(&sfull[sg & 1], (sg >> 1) & 1, LIMIT, abort_p)) return false;
                    }
                    const int at = (sg & 1) * C::G + kb % C::G;
                    f = make_float2(xsc[at * C::SROW + row], wsc[at * 2 + half]);
                    return true;
                });
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sempty[sg & 1]);
            if (!ok) break;
            store_rows<128>(args, (int64_t)(tile % MT) * 256 + rank * 128 + q * 32, tile / MT * 256 + col, sum,
                           smem + C::OUT + (warp - 4) * 4608, lane);
        }
    }
    if (!ok && lane == 0) fail();
    __syncthreads();
    if (*abort_p) {  // copies and MMAs in flight end before either CTA leaves
        if (warp == 2 && rank == 0 && tc::elect_one()) {
            int none = 0;
            tc::mma_commit_pair(drain, 1u);
            tc::mbar_wait(drain, 0, LIMIT / 100 + 100000, &none);
        }
        if (tid == 0) tc::wait_issued_fills(come, C::STAGES, *s_issued, LIMIT);
    }
    tc::tc_fence_before();
    __syncthreads();
    // (every arrival at the other CTA has been waited for there, unless a wait ran out: then they end here)
    if (*abort_p) tc::cluster_arrive_release();
    else tc::cluster_arrive();
    tc::cluster_wait();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Few rows of x.
// ---------------------------------------------------------------------------
namespace {

// NT: rows of x per tile.
template <int NT>
struct Narrow {
    static constexpr int EW = NT > 32 ? 8 : 4;  // warps that add blocks
    static constexpr int COLS = NT * 4 / EW;      // columns of each
    static constexpr int THREADS = 64 + 32 * EW;
    static constexpr int STAGE_BYTES = (128 + NT) * BK;
    static constexpr int STAGES = NT <= 16 ? 5 : NT <= 32 ? 4 : 3;  // and TMEM accumulators
    static constexpr int TMEM_COLS = STAGES * NT <= 128 ? 128 : 256;
    static constexpr int G = 32 * EW / NT;                 // blocks whose scales are fetched at a time, one per thread
    static constexpr int PITCH = 132;                      // row of a part: 128 weight rows and a gap (banks)
    static constexpr int SC_BASE = STAGES * STAGE_BYTES;   // scales [2][G][NT]
    static constexpr int RECV = SC_BASE + 2 * G * NT * 4;  // parts [split][rows / split][PITCH]
    static constexpr int BAR = RECV + (NT + 7) * PITCH * 4;
    static constexpr int BYTES = 1024 + BAR + 256;
    static_assert(NT * G == 32 * EW && STAGES * NT <= TMEM_COLS, "scale loads, accumulators");
    static_assert((2 * STAGES + 3) * 8 + 12 <= 256, "barrier area");
    static_assert(2 * (BYTES + 1024) <= 233472, "two CTAs on an SM");
    static_assert(NT * PITCH * 4 <= SC_BASE && RECV % 16 == 0, "a part fits over the ring");
};

}  // namespace

// Bound: the weights, once through HBM; from 32 rows on also what an SM takes in from L2, and the exchange. 1 row of
// 7168 x 9216 10.8 us (6.1 TB/s), 64 rows of 7168 x 7168 12.2 (4.3 TB/s). Two CTAs an SM: with 16 rows ten
// stages, 180 KB, on their way on each.
template <int NT>
__global__ void __launch_bounds__(Narrow<NT>::THREADS, 2)
    moe_linear_narrow_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX,
                             const MoeLinearArgs args) {
    using C = Narrow<NT>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *scales = (float *)(smem + C::SC_BASE), *parts = (float *)(smem + C::RECV);
    uint64_t *full = (uint64_t *)(smem + C::BAR);  // (barriers as in the kernel above)
    uint64_t *done = full + C::STAGES;
    uint64_t *recv = done + C::STAGES;
    uint64_t *drain = recv + 1;
    uint64_t *never = drain + 1;
    uint32_t *tmem_slot = (uint32_t *)(never + 1);
    int *abort_flag = (int *)(tmem_slot + 1);
    int *s_issued = abort_flag + 1;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int KB = (args.K + BK - 1) / BK, NTILES = (args.N + 127) / 128;
    const int rank = (int)tc::cluster_rank(), S = (int)tc::cluster_size(), tile = blockIdx.x / S;
    const int n0 = tile % NTILES * 128, t0 = tile / NTILES * NT;
    const int kb0 = KB * rank / S, nkb = KB * (rank + 1) / S - kb0;
    const int rows = min(NT, args.T - t0);
    // rows of x that a CTA joins, that this one does
    const int per = (rows + S - 1) / S, mine = min(per, rows - rank * per);
    if (tid == 0) {
        *abort_flag = 0;
        *s_issued = 0;
        for (int s = 0; s < C::STAGES; ++s) {
            tc::mbar_init(&full[s], 1 + C::EW);
            tc::mbar_init(&done[s], 1);
        }
        tc::mbar_init(recv, 1);
        tc::mbar_init(drain, 1);
        tc::mbar_init(never, 1);
        tc::fence_mbar_init();
        if (S > 1 && mine > 0) tc::mbar_arrive_expect_tx(recv, (S - 1) * mine * C::PITCH * 4);
        tc::prefetch_map(&mW);
        tc::prefetch_map(&mX);
        // the first stages' weights on their way to L2 while the kernel before ends
        for (int kb = 0; kb < min(C::STAGES, nkb); ++kb) tc::tma_prefetch_2d(&mW, (kb0 + kb) * BK, n0);
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (S > 1) tc::cluster_arrive();  // (1: this CTA's barriers are ready)
    const uint32_t tmem = *tmem_slot;
    const long long LIMIT = args.timeout_cycles;
    volatile int *abort_p = abort_flag;
    auto fail = [&](void) {
        *abort_p = 1;
        moe_flag(args.status, MOE_ERR_DEVICE_TIMEOUT);
    };
    grid_dep_wait();
    grid_dep_launch();
    bool ok = true;
    int drained = 0;
    if (warp == 0) {
        const uint64_t once = args.T <= NT ? tc::policy_evict_first() : tc::policy_evict_last();
        const uint64_t keep = tc::policy_evict_last();
        int it = 0;
        Ring at;
        for (; it < nkb; ++it, at.next(C::STAGES)) {
            if (it >= C::STAGES && !tc::mbar_wait_warp(&done[at.s], at.par ^ 1u, LIMIT, abort_p)) {
                ok = false;
                break;
            }
            if (tc::elect_one()) {
                unsigned char *st = smem + at.s * C::STAGE_BYTES;
                tc::mbar_arrive_expect_tx(&full[at.s], (uint32_t)C::STAGE_BYTES);
                tc::tma_load_2d(st, &mW, &full[at.s], (kb0 + it) * BK, n0, once);
                tc::tma_load_2d(st + 128 * BK, &mX, &full[at.s], (kb0 + it) * BK, t0, keep);
            }
            __syncwarp();
        }
        if (lane == 0) *s_issued = it;
    } else if (warp == 1) {
        const bool stall = stalls(args.inject, rank, S);
        Ring at;
        for (int it = 0; it < nkb; ++it, at.next(C::STAGES)) {
            if (!tc::mbar_wait_warp(&full[at.s], at.par, LIMIT, abort_p) ||
                (stall && !tc::mbar_wait_warp(never, 0, LIMIT, abort_p))) {
                ok = false;
                break;
            }
            tc::tc_fence_after();
            if (tc::elect_one()) {
                const uint32_t a_s = tc::smem_u32(smem) + at.s * C::STAGE_BYTES;
                mma_block<NT>(tmem + at.s * NT, a_s, a_s + 128 * BK);
                tc::mma_commit(&done[at.s]);
            }
            __syncwarp();
        }
        // (the last MMAs have finished when the adding warps are through with the last block)
    } else {
        const int q = warp & 3, row = q * 32 + lane, et = tid - 64;  // TMEM lane quadrant; weight row
        const int col0 = (warp - 2) / 4 * C::COLS;  // its first column
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + col0;
        const float *ws = args.w_s + (int64_t)(n0 / 128) * KB + kb0;
        if (lane == 0)
            for (int s = 0; s < C::STAGES; ++s) tc::mbar_arrive(&full[s]);  // (empty accumulators)
        // entry et of a group of scales: row et % NT of x, block et / NT (multiplied when stored, so that the
        // loads are in flight over the blocks before)
        float next, nextw;
        auto fetch = [&](int g) {
            const int r = et % NT, kb = g + et / NT;
            const bool in = r < rows && kb < nkb;
            next = in ? args.x_s[(t0 + r) * args.x_s_stride + kb0 + kb] : 0.f;
            nextw = in ? ws[kb] : 0.f;
        };
        fetch(0);
        float2 sum[C::COLS / 2];
#pragma unroll
        for (int j = 0; j < C::COLS / 2; ++j) sum[j] = make_float2(0.f, 0.f);
        Ring at;
        for (int it = 0; it < nkb; ++it, at.next(C::STAGES)) {
            const int g = it / C::G;
            float *sc = scales + (g & 1) * C::G * NT;
            if (it % C::G == 0) {
                // (two groups back: every warp is behind the barrier of the group between)
                sc[et] = next * nextw;
                fetch((g + 1) * C::G);
                asm volatile("bar.sync 1, %0;" ::"n"(32 * C::EW) : "memory");
            }
            // (a warp that gives up goes on to the barriers of the groups)
            if (ok && !tc::mbar_wait_warp(&done[at.s], at.par, LIMIT, abort_p)) ok = false;
            if (!ok) continue;
            tc::tc_fence_after();
            const float *f = sc + it % C::G * NT + col0;
            uint32_t r[C::COLS / 16][16];
#pragma unroll
            for (int h = 0; h < C::COLS / 16; ++h) tc::tmem_ld_32x32b_x16(acc + at.s * NT + 16 * h, r[h]);
            tc::tmem_ld_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&full[at.s]);
            ++drained;
#pragma unroll
            for (int j = 0; j < C::COLS; j += 4) {
                const float4 x = *(const float4 *)(f + j);
                fma2(sum[j / 2], r[j / 16][j % 16], r[j / 16][j % 16 + 1], x.x, x.y);
                fma2(sum[j / 2 + 1], r[j / 16][j % 16 + 2], r[j / 16][j % 16 + 3], x.z, x.w);
            }
        }
        if (S > 1) {
            if (ok) {  // over the ring, all of whose copies and MMAs are done
                float *o = (float *)smem + col0 * C::PITCH + row;
#pragma unroll
                for (int j = 0; j < C::COLS; ++j)
                    if (col0 + j < rows) o[j * C::PITCH] = j & 1 ? sum[j / 2].y : sum[j / 2].x;
            }
            tc::fence_proxy_async_smem();
            ok = tc::bar_and(1, 32 * C::EW, ok);
        } else if (ok && n0 + row < args.N) {
            const int64_t to = (int64_t)(t0 + col0) * args.out_stride + n0 + row;
#pragma unroll
            for (int j = 0; j < C::COLS; ++j)
                if (col0 + j < rows) store1(args, to + j * args.out_stride, j & 1 ? sum[j / 2].y : sum[j / 2].x);
        }
    }
    if (!ok && lane == 0) fail();
    __syncwarp();
    if (S > 1) {
        tc::cluster_wait();  // (1)
        if (warp >= 2) {
            if (warp == 2) send_parts((const float *)smem, parts, recv, S, rank, rows, per, C::PITCH, lane);
            if (mine > 0 && !wait_parts(recv, KB, LIMIT)) ok = false;
            if (!ok && lane == 0) fail();
            __syncwarp();
        }
        if (warp >= 2 && ok) {
            for (int u = tid - 64; u < mine * 32; u += 32 * C::EW) {
                const int j = u / 32, n = n0 + u % 32 * 4;
                if (n < args.N)
                    store4(args, (int64_t)(t0 + rank * per + j) * args.out_stride + n,
                           join((const float *)smem + (rank * per + j) * C::PITCH + u % 32 * 4,
                                parts + j * C::PITCH + u % 32 * 4, per * C::PITCH, rank, S));
            }
        }
        __syncwarp();
        // (2: this CTA has the parts of its rows. Behind the join, so that the CTAs of a cluster leave together: ahead of
        // it those with few rows or none leave early, and where as many of the next kernel's clusters are wanted as fit,
        // the last ones find no room until the others have left: 1 row of 7168 x 7168 by 5 10.8 us, 3 rows 10.0, so
        // 9.0 both; where all find room in any case up to 0.1 us less, 1 row of 7168 x 9216 10.8 and 10.85.)
        tc::cluster_arrive();
        tc::cluster_wait();  // (2: all parts have arrived, also where a wait ran out: none is on its way to or from here)
    }
    __syncthreads();
    if (*abort_p) wind_down<C::STAGES>(full, drain, warp == 1, warp >= 2 && lane == 0, drained, *s_issued, LIMIT);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

namespace {

// Which kernel, and the CTAs (up to 8) that share a tile's K. Times of both sides in us.
//   Few rows: the split of the least cost, of blocks per CTA (0.2 us each), the exchange (0.25, 0.02 a CTA) and two
//   CTAs on an SM (0.35, where they are on a few SMs only 0.3 more). 1 row of 7168 x 9216 (72 tiles): by 1 15.0, 2
//   12.6, 3 11.8, 4 10.8; of 7168 x 5632 (44): by 4 8.9, 6 7.5; of 2048 x 4096 (32): by 4 3.7, 8 4.0; of 4096 x 4096:
//   by 4 5.6, 8 5.0; 64 rows of 2048 x 2048 (16): by 6 5.1, 8 5.8; of 256 x 2048: by 1 3.8, 2 4.2. All clusters have
//   to fit beside each other: 1 row of 7168 x 9600 (75) by 4 15.8, by 3 12.1.
//   Rows per tile: all, or fewer where more tiles find SMs to run on, up to 256 rows or so of few weights; both
//   kernels' times are estimated, and a change has to win 8 or 10 in a hundred. 64 rows of 1040 x 776: tiles of 64 4.7,
//   of 16 3.4; of 4096 x 5120: 9.0 and 10.6. 128 rows of 4096 x 1000: tiles of 32 5.6, of 128 (the other kernel) 8.0;
//   of 4096 x 4096 10.0 and 9.7; 256 rows of 7168 x 264: tiles of 64 6.9, of 128 8.4.
//   Many rows: the exchange of a 128 x 128 part costs about 2 us, so K is split where that saves more (128 rows of
//   4096 x 5120 (40 tiles): by 1 13.2, 2 11.9, 3 10.6, but of 2048 x 6144 (48) by 1 8.5, 2 9.4; of 2048 x 2816 (22) by
//   4 8.0, by 6 8.1, of 4096 x 2816 9.2 and 9.0), and only by as many as fit (1000 columns of 4096: 128 rows (8 tiles)
//   by 4 8.4, by 8 7.9; 200 rows (16) by 6 8.3, by 8 11.8; 384 rows (24) by 4 8.9, by 6 15.1).
//   Very many: by the times that the two kernels' waves take, which these sizes gave (waves of the many-row kernel
//   and of pairs, times of both): 512 rows of 7168 x 9216 2, 1, 37.3, 28.1; 600 rows 3, 2, 50.6, 48.7; 8191 rows
//   31, 16, 482, 384; 900 rows of 4096 x 5120 3, 2, 29.6, 31.3; 2049 rows 5, 3, 47.6, 45.9; 768 rows of 1536 x 7168
//   3, 2, 14.9, 16.9; 4096 rows 12, 6, 47.8, 43.5. (The ns a block and a tile in the rules are fitted to whole calls; a
//   block alone takes 306 ns in the many-row kernel, 375 in the pairs'.)
struct Plan {
    int nt;     // rows of x per tile of the few-row kernel; 0: the others
    bool pair;  // the CTA pairs' kernel
    int split;
};

// Clusters of s CTAs that 152 SMs hold at a time with one CTA an SM (the occupancy query's answers), and with two
// (found by the few-row kernel's times: that query counts one of these CTAs an SM).
constexpr int kClusters1[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
constexpr int kClusters2[9] = {0, 304, 152, 92, 72, 56, 46, 38, 36};

// Split (0: too many tiles for tiles of less than all rows) and about the time, ns, of the few-row kernel with tiles of
// nt rows. What a block takes is what it moves through shared memory, so two CTAs on an SM take nearly twice as long.
struct Few {
    int split;
    int64_t ns;
};

Few few_rows(int nt, int T, int K, int N, int nsm) {
    const int KB = (K + BK - 1) / BK, i = nt == 16 ? 0 : nt == 32 ? 1 : 2;
    const int64_t tiles = (int64_t)((N + 127) / 128) * ((T + nt - 1) / nt), clusters = tiles * 152;
    if (T > nt && clusters > (int64_t)kClusters2[1] * nsm) return {0, 0};
    Few few = {1, 0};
    for (int s = 1, least = INT32_MAX; s <= 8 && KB >= s; ++s) {
        if (s > 1 && clusters > (int64_t)kClusters2[s] * nsm) continue;
        const int nb = (KB + s - 1) / s;
        const bool two = clusters > (int64_t)kClusters1[s] * nsm, uneven = two && tiles * s * 4 < 5 * nsm;
        const int cost = 200 * nb + 20 * s + 250 * (s > 1) + 350 * two + 300 * uneven;
        if (cost >= least) continue;
        constexpr int start[3] = {2300, 2750, 3200}, block[2][3] = {{215, 275, 340}, {225, 320, 510}};
        least = cost;
        few = {s, start[i] + 550 * (s > 1) + 800 * two + (int64_t)nb * block[two][i]};
    }
    return few;
}

Plan plan_of(int T, int K, int N, int nsm) {
    const int KB = (K + BK - 1) / BK;
    if (T <= 64) {
        int nt = T <= 16 ? 16 : T <= 32 ? 32 : 64;
        Few best = few_rows(nt, T, K, N, nsm);
        for (int low = 16, all = nt, most = (int)(best.ns * 100 / 108); low < all; low *= 2) {
            const Few few = few_rows(low, T, K, N, nsm);
            if (few.split > 0 && few.ns < most) best = few, nt = low, most = (int)few.ns;
        }
        return {nt, false, best.split};
    }
    const int64_t mt = (T + 127) / 128, tiles = (N + 127) / 128 * mt;
    const int64_t pairs = (int64_t)((N + 255) / 256) * ((T + 255) / 256);
    int s = 1;
    if (KB >= 16 && tiles * 8 <= nsm * 3 / 4) s = 8;
    else if (KB >= 32 && tiles * 6 <= nsm * 7 / 8) s = 6;
    else if (KB >= 16 && tiles * 4 <= nsm * 15 / 16) s = 4;
    else if (KB >= 20 && tiles * 3 <= nsm * 7 / 8) s = 3;
    else if (KB >= 24 && tiles * 2 <= nsm) s = 2;
    if (tiles <= nsm) {
        const int64_t rows = T / mt, wide = 1700 + 360 * ((KB + s - 1) / s) + (s > 1) * (1250 + rows * 2100 / 128) + rows * 1700 / 128;
        Plan plan = {0, false, 0};
        for (int64_t nt = 16, most = wide * 10 / 11; nt <= 64; nt *= 2) {
            const Few few = few_rows((int)nt, T, K, N, nsm);
            const int64_t ns = few.ns + (int64_t)K * N / 27000;  // (and the weights' way from HBM)
            if (few.split > 0 && ns < most) plan = {(int)nt, false, few.split}, most = ns;
        }
        if (plan.nt > 0) return plan;
    }
    const int64_t waves = (tiles + nsm - 1) / nsm, pair_waves = (pairs + nsm / 2 - 1) / (nsm / 2);
    const bool pair = 5500 + pair_waves * (365 * KB + 1100) < 4000 + waves * (265 * KB + 400);  // ns
    return {0, pair, pair ? 1 : s};
}

template <typename... KArgs>
cudaError_t launch_split(void (*kern)(KArgs...), int64_t grid, int threads, int smem, int split, cudaStream_t st,
                         const CUtensorMap &map_w, const CUtensorMap &map_x, const MoeLinearArgs &a) {
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, map_w, map_x, a);
}

template <int NT>
cudaError_t launch_narrow(int split, cudaStream_t st, const CUtensorMap &w, const CUtensorMap &x,
                          const MoeLinearArgs &a) {
    const int64_t tiles = (int64_t)((a.N + 127) / 128) * ((a.T + NT - 1) / NT);
    return launch_split(moe_linear_narrow_kernel<NT>, tiles * split, Narrow<NT>::THREADS, Narrow<NT>::BYTES, split, st, w,
                        x, a);
}

cudaError_t launch_wide(int split, int nsm, cudaStream_t st, const CUtensorMap &w, const CUtensorMap &x,
                        const MoeLinearArgs &a) {
    const int64_t tiles = (int64_t)((a.T + 127) / 128) * ((a.N + 127) / 128);
    return launch_split(moe_linear_wide_kernel, split > 1 ? tiles * split : tiles < nsm ? tiles : nsm, Wide::THREADS,
                        Wide::BYTES, split, st, w, x, a);
}

cudaError_t launch_pair(int nsm, cudaStream_t st, const CUtensorMap &w, const CUtensorMap &x, const MoeLinearArgs &a) {
    const int64_t tiles = (int64_t)((a.T + 255) / 256) * ((a.N + 255) / 256), pairs = nsm / 2;
    return launch_split(moe_linear_pair_kernel, 2 * (tiles < pairs ? tiles : pairs), Pair::THREADS, Pair::BYTES, 2, st, w,
                        x, a);
}

}  // namespace

cudaError_t moe_linear_setup() {
    cudaError_t err = set_kernel((const void *)moe_linear_wide_kernel, Wide::BYTES);
    if (err == cudaSuccess) err = set_kernel((const void *)moe_linear_pair_kernel, Pair::BYTES);
    if (err == cudaSuccess) err = set_kernel((const void *)moe_linear_narrow_kernel<16>, Narrow<16>::BYTES);
    if (err == cudaSuccess) err = set_kernel((const void *)moe_linear_narrow_kernel<32>, Narrow<32>::BYTES);
    if (err == cudaSuccess) err = set_kernel((const void *)moe_linear_narrow_kernel<64>, Narrow<64>::BYTES);
    // the pair's register split waits forever if the kernel was built with fewer
    cudaFuncAttributes f;
    if (err == cudaSuccess) err = cudaFuncGetAttributes(&f, (const void *)moe_linear_pair_kernel);
    if (err == cudaSuccess && f.numRegs != Pair::REGS) err = cudaErrorInvalidKernelImage;
    return err;
}

MoeLinearBox moe_linear_box(int T, int K, int N, int nsm) {
    const Plan p = plan_of(T, K, N, nsm);
    return {p.nt > 0 ? p.nt : 128, p.pair};
}

cudaError_t moe_launch_linear(const CUtensorMap &map_w, const CUtensorMap &map_x, const MoeLinearArgs &a, int nsm,
                              cudaStream_t st) {
    const Plan p = plan_of(a.T, a.K, a.N, nsm);
    switch (p.nt) {
        case 16: return launch_narrow<16>(p.split, st, map_w, map_x, a);
        case 32: return launch_narrow<32>(p.split, st, map_w, map_x, a);
        case 64: return launch_narrow<64>(p.split, st, map_w, map_x, a);
    }
    return p.pair ? launch_pair(nsm, st, map_w, map_x, a) : launch_wide(p.split, nsm, st, map_w, map_x, a);
}
