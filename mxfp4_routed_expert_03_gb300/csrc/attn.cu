// Attention over the MXFP4 key/value cache (moe_attn_forward).
//
// One pass over the keys with a running maximum m and sum l per query row:
//   s = scale log2(e) q.k,  m' = max(m, s),  p = 2^(s - m'),
//   l = l 2^(m - m') + sum p,  o = o 2^(m - m') + sum p v,
// out = o / l, lse = ln2 (m + log2 l).
//
// Shape of the work. The query heads that share a key/value head, times the
// query rows of a sequence, are the columns of small matrix products with the
// cache as the other operand: S^T = K Q^T (16 tokens x 8 columns x 16
// dimensions per mma.sync) and O^T = V^T P^T. Tokens sit on the 16-wide side,
// so 8 columns (a decode step of a group of 8 heads) waste nothing.
//
// Codes to operands. The cache keeps 8 tokens x 32 dimensions as an 8x8 tile
// of 16-bit units (4 codes each): ldmatrix gives a lane 8 codes of one token,
// which are 4 fp16 pairs of a K fragment (cvt e2m1x2 -> f16x2); its transposed
// form gives 4 codes of two neighbouring tokens, which one byte permute per
// pair turns into the V fragment (tokens are the contracted index there). The
// codes are exact in fp16; scales never touch them: a key block's scale
// multiplies the block's partial product in fp32, a value block's scale goes
// into the weight p, as 2^(e - R) with R a running maximum of the block's
// exponents (o carries 2^R), so p 2^(e - R) stays within fp16 (values over
// 2^29 below the largest vanish). p itself is rounded to fp16 (11 bits).
// Queries are put into fp16 with one power of two per row, exact for elements
// within 2^-29 of the row's largest.
//
// Split. Tokens go in tiles of 32; all (sequence, column tile, head) items'
// tiles form one line that is cut into equal pieces, one per CTA, so any mix
// of lengths is balanced. A CTA's 4 warps take a piece's tiles in turn, each
// with its own ring of bulk copies and its own m, l, o, and merge at the end;
// items cut between CTAs leave partial results that a second kernel joins in
// a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kTile = 32;      // tokens per tile
constexpr int kStages = 3;     // tiles in flight per warp
constexpr int kMinTiles = 4;   // per CTA: one for each warp
constexpr uint32_t kFull = 0xFFFFFFFFu;

template <int D, int NT>
struct Cfg {
    static constexpr int NB = D / 32;             // blocks of a head row
    static constexpr int NC = 8 * NT;             // columns of a tile
    static constexpr int kCode = kTile * D / 2;   // bytes of a tile's K (or V) codes
    static constexpr int kScale = kTile * NB;
    static constexpr int kStage = 2 * (kCode + kScale);
    static constexpr int kOStride = D + 4;
    static constexpr int kSmemO = kWarps * kStages * kStage;
    static constexpr int kSmemMl = kSmemO + kWarps * NC * kOStride * 4;
    static constexpr int kSmemBar = kSmemMl + 2 * kWarps * NC * 4;
    static constexpr int kSmem = kSmemBar + kWarps * kStages * 8 + kWarps * kStages * 4 + 64;
    static constexpr int kCtasPerSm = NT == 1 ? 3 : 2;
    static constexpr int kRec = NC * (D + 2);     // floats of a partial result: o, m, l
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
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
__device__ __forceinline__ void bulk_g2s(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            tc::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ float pow2(int e) {  // 2^e for e in [-127, 127]
    return __uint_as_float(e == -127 ? 0x00400000u : (uint32_t)(e + 127) << 23);
}

// ------------------------------------------------------------------ schedule
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

// Units of the line: token tiles, or whole items where max_kv is short.
template <int NC>
__device__ __forceinline__ long long seq_work(const MoeAttnArgs &a, int b, bool whole) {
    const Seq s = seq_of<NC>(a, b);
    return (long long)s.cts * a.n_kv * (whole ? 1 : s.tiles);
}

// Sum of v over the block's 4 warps (all threads get it) and each thread's
// inclusive prefix; tot: 4 words of shared memory.
__device__ __forceinline__ long long block_scan(long long v, long long *tot, long long &incl) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += o;
    }
    __syncthreads();
    if (lane == 31) tot[wid] = incl;
    __syncthreads();
    long long sum = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == wid) before = sum;
        sum += tot[w];
    }
    incl += before;
    return sum;
}

// Units of all sequences.
template <int NC>
__device__ long long total_work(const MoeAttnArgs &a, bool whole, long long *tot) {
    long long w = 0;
    for (int base = 0; base < a.b.n_seqs; base += 32 * kWarps) {
        const int b = base + threadIdx.x;
        long long incl;
        w += block_scan(b < a.b.n_seqs ? seq_work<NC>(a, b, whole) : 0, tot, incl);
    }
    return w;
}

// The sequence that holds unit `pos` (0 <= pos < total) and the unit's offset
// in it; res: 2 words of shared memory.
template <int NC>
__device__ void find_unit(const MoeAttnArgs &a, bool whole, long long pos, long long *tot,
                          long long *res, int &seq, long long &off) {
    long long before = 0;
    for (int base = 0; base < a.b.n_seqs; base += 32 * kWarps) {
        const int b = base + threadIdx.x;
        const long long v = b < a.b.n_seqs ? seq_work<NC>(a, b, whole) : 0;
        long long incl;
        const long long sum = block_scan(v, tot, incl);
        if (pos < before + sum) {  // block-uniform
            const long long first = before + incl - v;
            if (pos >= first && pos < first + v) {
                res[0] = b;
                res[1] = pos - first;
            }
            break;
        }
        before += sum;
    }
    __syncthreads();
    seq = (int)res[0];
    off = res[1];
    __syncthreads();
}

// Units per CTA.
__device__ __forceinline__ long long piece_of(long long total, int ctas, bool whole) {
    const long long per = (total + ctas - 1) / ctas;
    return whole ? (per > 0 ? per : 1) : (per > kMinTiles ? per : kMinTiles);
}

// Output of one column: o / l, or 0 where no key was seen.
__device__ __forceinline__ void store_row(const MoeAttnArgs &a, int row, int d, float o0, float o1,
                                          float l) {
    const float r = l == 0.f ? 0.f : 1.f / l;
    const __nv_bfloat162 v = __floats2bfloat162_rn(l == 0.f ? 0.f : o0 * r, l == 0.f ? 0.f : o1 * r);
    *(__nv_bfloat162 *)(a.out + (int64_t)row * a.out_stride + d) = v;
}

// ------------------------------------------------------------------ kernel
template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, Cfg<D, NT>::kCtasPerSm)
    moe_attn_split_kernel(MoeAttnArgs a, bool whole) {
    using C = Cfg<D, NT>;
    constexpr int NB = C::NB, NC = C::NC;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_tot[kWarps], s_res[2];
    __shared__ int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem + wid * kStages * C::kStage;
    float *s_o = (float *)(smem + C::kSmemO);
    float *s_m = (float *)(smem + C::kSmemMl), *s_l = s_m + kWarps * NC;
    uint64_t *full = (uint64_t *)(smem + C::kSmemBar) + wid * kStages;
    uint32_t *valid = (uint32_t *)(smem + C::kSmemBar + kWarps * kStages * 8) + wid * kStages;
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) tc::mbar_init(&full[i], 1);
    if (tid == 0) s_abort = 0;
    tc::fence_mbar_init();
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();

    const long long total = total_work<NC>(a, whole, s_tot);
    const long long per = piece_of(total, gridDim.x, whole);
    long long pos = blockIdx.x * per;
    const long long end = min(total, pos + per);
    if (pos >= end) return;
    int b;
    long long off;
    find_unit<NC>(a, whole, pos, s_tot, s_res, b, off);

    uint32_t fills = 0, uses = 0;  // of this warp's ring, over all items
    bool dead = false;             // a wait ran out: no more copies or waits
    const int parts = a.page_shift == 4 ? 2 : 1;  // pages of a tile
    const int ids_cap = 32 / parts;               // tiles whose page ids a warp holds

    while (pos < end) {
        const Seq s = seq_of<NC>(a, b);
        const int units = whole ? 1 : s.tiles;
        const long long items = (long long)s.cts * a.n_kv;
        if (items == 0 || off >= items * units) {  // no rows, or past the sequence's last item
            ++b;
            off = 0;
            continue;
        }
        const int item = (int)(off / units), u0 = (int)(off % units);
        const int take = (int)min((long long)(units - u0), end - pos);
        const int tb = whole ? 0 : u0, te = whole ? s.tiles : u0 + take;
        const bool starts = u0 == 0, ends = u0 + take == units;
        const int ct = item / a.n_kv, h = item % a.n_kv;
        const int c0 = ct * NC;
        const int i0 = c0 / a.group, i1 = (min(c0 + NC, s.ncol) - 1) / a.group;
        const int p0 = s.kv - s.nq;                 // position of query row 0
        const int hi_max = p0 + i1 + 1, hi_min = p0 + i0 + 1;  // key bounds over the columns
        const int lo_min = a.b.window > 0 ? max(0, hi_min - a.b.window) : 0;
        const int lo_max = a.b.window > 0 ? max(0, hi_max - a.b.window) : 0;
        const int x_lo = max(tb, (lo_min - s.lo) / kTile);
        const int x_hi = hi_max <= s.lo ? 0 : min(te, (hi_max - s.lo + kTile - 1) / kTile);
        const int n_my = x_hi - x_lo > wid ? (x_hi - x_lo - wid + kWarps - 1) / kWarps : 0;

        // --- queries: fp16 with one power of two per column, and key bounds
        uint32_t qf[NT][NB][4];
        float mul[NT][2];       // of columns 2t, 2t + 1: back from that power of two, scale log2(e)
        int hi[NT][2], lo[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int c = c0 + 8 * n + g;
            uint4 raw[NB];
            uint32_t top = 0u;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                raw[k] = make_uint4(0u, 0u, 0u, 0u);
                if (c < s.ncol)
                    raw[k] = *(const uint4 *)(a.q + (int64_t)(s.q0 + c / a.group) * a.q_stride +
                                              (h * a.group + c % a.group) * D + 32 * k + 8 * t);
                top = __vmaxu2(top, raw[k].x & 0x7FFF7FFFu);
                top = __vmaxu2(top, raw[k].y & 0x7FFF7FFFu);
                top = __vmaxu2(top, raw[k].z & 0x7FFF7FFFu);
                top = __vmaxu2(top, raw[k].w & 0x7FFF7FFFu);
            }
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(kFull, top, 1));
            top = max(top, __shfl_xor_sync(kFull, top, 2));
            // largest magnitude to [2^14, 2^15); a row with an infinity or NaN
            // gets a NaN factor
            const int sh = min(141 - (int)(top >> 7), 127);
            const float up = __uint_as_float((uint32_t)(sh + 127) << 23);
            const float down = top >= 0x7F80u ? CUDART_NAN_F : pow2(-sh);
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    qf[n][k][j] = pack_f16(__uint_as_float(w[j] << 16) * up,
                                           __uint_as_float(w[j] & 0xFFFF0000u) * up);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int cc = c0 + 8 * n + 2 * t + j;
                mul[n][j] = __shfl_sync(kFull, down, 4 * (2 * t + j)) * (a.b.scale * CUDART_L2E_F);
                hi[n][j] = cc < s.ncol ? p0 + cc / a.group + 1 : 0x7FFFFFFF;
                lo[n][j] = cc < s.ncol && a.b.window > 0 ? hi[n][j] - a.b.window : 0;
            }
        }

        float o[NB][2][NT][4], m[NT][2], l[NT][2];
        uint32_t R[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            R[k] = 0u;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[k][hh][n][c] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;

        // --- ring: the warp's tile j covers tokens first + 32 * 4 * j ..
        const int first = s.lo + kTile * (x_lo + wid);
        int ids = -1;
        auto issue = [&](int j) {
            const int part = parts == 2 ? lane & 1 : 0;
            if (j % ids_cap == 0) {  // page ids of the next tiles, a lane each
                const int jj = j + (parts == 2 ? lane >> 1 : lane);
                const int tok = first + kTile * kWarps * jj + 16 * part;
                ids = -2;  // no token of that page is needed
                if (jj < n_my && tok < hi_max) {
                    ids = a.b.page_table[(int64_t)b * a.b.table_stride + (tok >> a.page_shift)];
                    if (ids < 0 || ids >= a.n_pages) {
                        moe_flag(a.status, MOE_ERR_BAD_INDEX);
                        ids = -1;
                    }
                }
            }
            const int at = (j % ids_cap) * parts;
            const int id0 = __shfl_sync(kFull, ids, at);
            const int id1 = parts == 2 ? __shfl_sync(kFull, ids, at + 1) : id0;
            const int st = fills % kStages;
            uint8_t *dst = ring + st * C::kStage;
            const int ok0 = id0 >= 0, ok1 = parts == 2 && id1 >= 0;
            const uint32_t half = C::kStage / parts;
            if (lane == 0) {
                valid[st] = parts == 2 ? (ok0 ? 0xFFFFu : 0u) | (ok1 ? 0xFFFF0000u : 0u)
                                       : (ok0 ? kFull : 0u);
                tc::mbar_arrive_expect_tx(&full[st], (ok0 + ok1) * half);
            }
            __syncwarp();
            // lane 0..3 (and 4..7): K codes, V codes, K scales, V scales of a page
            const int which = lane & 3, pt = lane >> 2;
            const int id = pt ? id1 : id0;
            if (lane < 4 * parts && id >= 0) {
                const int tok = first + kTile * kWarps * j + 16 * pt;
                const int64_t row = (((int64_t)id * a.n_kv + h) << a.page_shift) +
                                    (tok & ((1 << a.page_shift) - 1));
                const uint8_t *src = which == 0   ? a.c.k_q + row * (NB * 16)
                                     : which == 1 ? a.c.v_q + row * (NB * 16)
                                     : which == 2 ? a.c.k_s + row * NB
                                                  : a.c.v_s + row * NB;
                const int bytes = (which < 2 ? C::kCode : C::kScale) / parts;
                uint8_t *to = dst + (which < 2 ? which * C::kCode
                                               : 2 * C::kCode + (which - 2) * C::kScale) + pt * bytes;
                bulk_g2s(to, src, bytes, &full[st]);
            }
            ++fills;
        };
        if (!dead)
            for (int j = 0; j < kStages && j < n_my; ++j) issue(j);

        for (int j = 0; j < n_my && !dead; ++j) {
            const int st = uses % kStages;
            const bool ok = tc::mbar_wait(&full[st], (uses / kStages) & 1, a.timeout_cycles, &s_abort);
            if (!__all_sync(kFull, ok)) {
                if (lane == 0) {
                    moe_flag(a.status, MOE_ERR_DEVICE_TIMEOUT);
                    s_abort = 1;
                }
                dead = true;
                break;
            }
            const uint32_t base = tc::smem_u32(ring + st * C::kStage);
            const uint8_t *ks = ring + st * C::kStage + 2 * C::kCode, *vs = ks + C::kScale;
            const int tok0 = first + kTile * kWarps * j;
            const uint32_t live = valid[st];
            const bool edge = tok0 + kTile > hi_min || tok0 < lo_max || live != kFull;

            // --- S^T = K Q^T of 2 x 16 tokens
            float sc[2][NT][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) sc[u][n][c] = 0.f;
                uint32_t w0, w1;  // scale bytes of tokens g and g + 8
                if constexpr (NB == 4) {
                    w0 = *(const uint32_t *)(ks + (16 * u + g) * 4);
                    w1 = *(const uint32_t *)(ks + (16 * u + g + 8) * 4);
                } else {
                    w0 = *(const uint16_t *)(ks + (16 * u + g) * 2);
                    w1 = *(const uint16_t *)(ks + (16 * u + g + 8) * 2);
                }
#pragma unroll
                for (int kk = 0; kk < NB / 2; ++kk) {
                    uint32_t r[4];  // (octet 0, 1) of block 2kk, then of block 2kk + 1
                    const int mat = lane >> 3;
                    ldsm4(r, base + ((2 * u + (mat & 1)) * NB + 2 * kk + (mat >> 1)) * 128 +
                                 (lane & 7) * 16);
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        const int k = 2 * kk + k2;
                        uint32_t ha[4], hb[4];
                        codes_f16(r[2 * k2], ha);
                        codes_f16(r[2 * k2 + 1], hb);
                        // 2^(byte - 127); the lowest bit set makes 255 a NaN
                        // (and is a 2^-23 error otherwise)
                        const uint32_t e0 = k == 0 ? w0 << 23 : k == 1 ? w0 << 15 : k == 2 ? w0 << 7 : w0 >> 1;
                        const uint32_t e1 = k == 0 ? w1 << 23 : k == 1 ? w1 << 15 : k == 2 ? w1 << 7 : w1 >> 1;
                        const float f0 = __uint_as_float((e0 & 0x7F800000u) | 1u);
                        const float f1 = __uint_as_float((e1 & 0x7F800000u) | 1u);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float c[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_f16(c, ha[0], hb[0], ha[1], hb[1], qf[n][k][0], qf[n][k][1]);
                            mma_f16(c, ha[2], hb[2], ha[3], hb[3], qf[n][k][2], qf[n][k][3]);
                            sc[u][n][0] = fmaf(c[0], f0, sc[u][n][0]);
                            sc[u][n][1] = fmaf(c[1], f0, sc[u][n][1]);
                            sc[u][n][2] = fmaf(c[2], f1, sc[u][n][2]);
                            sc[u][n][3] = fmaf(c[3], f1, sc[u][n][3]);
                        }
                    }
                }
            }
            // --- running maximum
            bool grew = false;
            float mx[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = -INFINITY;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float &x = sc[u][n][2 * r + c];
                            x *= mul[n][c];
                            if (edge) {
                                const int i = 16 * u + 8 * r + g, tk = tok0 + i;
                                if (tk >= hi[n][c] || tk < lo[n][c] || !((live >> i) & 1u))
                                    x = -INFINITY;
                            }
                            v = fmaxf(v, x);
                        }
                    v = fmaxf(v, __shfl_xor_sync(kFull, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(kFull, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(kFull, v, 16));
                    mx[n][c] = fmaxf(m[n][c], v);
                    grew |= mx[n][c] > m[n][c];
                }
            if (__any_sync(kFull, grew)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float f = mx[n][c] == -INFINITY ? 1.f : ex2(m[n][c] - mx[n][c]);
                        m[n][c] = mx[n][c];
                        l[n][c] *= f;
#pragma unroll
                        for (int k = 0; k < NB; ++k)
#pragma unroll
                            for (int hh = 0; hh < 2; ++hh) {
                                o[k][hh][n][c] *= f;
                                o[k][hh][n][c + 2] *= f;
                            }
                    }
            }
            // --- O^T += V^T P^T, 16 tokens at a time
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t pt[NT][2];  // weights of tokens (2t, 2t + 1) of octet 0, 1; column g
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float p[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float mm = m[n][c & 1];
                        p[c] = ex2(sc[u][n][c] - (mm == -INFINITY ? 0.f : mm));
                        l[n][c & 1] += p[c];
                    }
                    pt[n][0] = transpose8(pack_f16(p[0], p[1]));
                    pt[n][1] = transpose8(pack_f16(p[2], p[3]));
                }
                uint32_t v2[2][NB], d2[2][NB], any = 0u;  // exponents of tokens 2t, 2t + 1
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint8_t *src = vs + (4 * (2 * u + q) + t) * (2 * NB);
                    uint32_t keep = kFull;
                    if (edge) {  // tokens that no column sees must not set R
                        const int i = 16 * u + 8 * q + 2 * t, tk = tok0 + i;
                        const bool s0 = tk < hi_max && tk >= lo_min && ((live >> i) & 1u);
                        const bool s1 = tk + 1 < hi_max && tk + 1 >= lo_min && ((live >> (i + 1)) & 1u);
                        keep = (s0 ? 0xFFFFu : 0u) | (s1 ? 0xFFFF0000u : 0u);
                    }
#pragma unroll
                    for (int kk = 0; kk < NB / 2; ++kk) {
                        const uint32_t w = *(const uint32_t *)(src + 4 * kk);
                        v2[q][2 * kk] = __byte_perm(w, 0u, 0x4140) & keep;
                        v2[q][2 * kk + 1] = __byte_perm(w, 0u, 0x4342) & keep;
                    }
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        // e + 31 - R, at least 1; above 31 the running maximum is stale
                        d2[q][k] = __viaddmax_s16x2(v2[q][k], ((31u - R[k]) & 0xFFFFu) * 0x00010001u, 0x00010001u);
                        any |= d2[q][k];
                    }
                }
                bool special = false;  // a value scale that is NaN
                if (__any_sync(kFull, (any & 0x01E001E0u) != 0u)) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        uint32_t top = R[k];
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t x = (v2[q][k] >> (16 * e)) & 0xFFFFu;
                                if (x == 255u) special = true;
                                else top = max(top, x);
                            }
                        top = max(top, __shfl_xor_sync(kFull, top, 1));
                        top = max(top, __shfl_xor_sync(kFull, top, 2));
                        const float f = exp2f((float)((int)R[k] - (int)top));
                        R[k] = top;
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int c = 0; c < 4; ++c) o[k][hh][n][c] *= f;
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            d2[q][k] = __viaddmax_s16x2(v2[q][k], ((31u - R[k]) & 0xFFFFu) * 0x00010001u, 0x00010001u);
                    }
                    special = __any_sync(kFull, special);
                }
                uint32_t pv[NT][2][NB];  // weight x 2^(15 + e - R)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        const uint32_t f = d2[q][k] * 1024u - 0x04000400u;
#pragma unroll
                        for (int n = 0; n < NT; ++n) pv[n][q][k] = mul_f16x2(pt[n][q], f);
                        if (special) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t half = 0xFFFFu << (16 * e);
                                if (((v2[q][k] >> (16 * e)) & 0xFFFFu) == 255u) {
#pragma unroll
                                    for (int n = 0; n < NT; ++n) {
                                        pv[n][q][k] &= ~half;
                                        if (pt[n][q] & half) pv[n][q][k] |= 0x7E007E00u & half;
                                    }
                                }
                            }
                        }
                    }
#pragma unroll
                for (int kk = 0; kk < NB / 2; ++kk) {
                    uint32_t r[4];  // (octet 0, 1) of block 2kk, then of block 2kk + 1
                    const int mat = lane >> 3;
                    ldsm4_t(r, base + C::kCode +
                                   ((2 * u + (mat & 1)) * NB + 2 * kk + (mat >> 1)) * 128 +
                                   (lane & 7) * 16);
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        const int k = 2 * kk + k2;
                        uint32_t ha[4], hb[4];
                        codes_f16(r[2 * k2], ha);      // [0, 1]: token 2t, [2, 3]: token 2t + 1
                        codes_f16(r[2 * k2 + 1], hb);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const uint32_t a0 = __byte_perm(ha[hh], ha[hh + 2], 0x5410);
                            const uint32_t a1 = __byte_perm(ha[hh], ha[hh + 2], 0x7632);
                            const uint32_t a2 = __byte_perm(hb[hh], hb[hh + 2], 0x5410);
                            const uint32_t a3 = __byte_perm(hb[hh], hb[hh + 2], 0x7632);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16(o[k][hh][n], a0, a1, a2, a3, pv[n][0][k], pv[n][1][k]);
                        }
                    }
                }
            }
            ++uses;
            __syncwarp();
            if (j + kStages < n_my) issue(j + kStages);
        }

        // --- the 4 warps' results: o, m, l of each column
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = l[n][c];
                v += __shfl_xor_sync(kFull, v, 4);
                v += __shfl_xor_sync(kFull, v, 8);
                v += __shfl_xor_sync(kFull, v, 16);
                const int col = 8 * n + 2 * t + c;
                if (g == 0) {
                    s_m[wid * NC + col] = m[n][c];
                    s_l[wid * NC + col] = v;
                }
                float *dst = s_o + (wid * NC + col) * C::kOStride + 4 * g;
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    const float f = exp2f((float)((int)R[k] - 142));  // 2^(R - 127) / 2^15
                    *(float4 *)(dst + 32 * k) =
                        make_float4(o[k][0][n][c] * f, o[k][0][n][c + 2] * f, o[k][1][n][c] * f,
                                    o[k][1][n][c + 2] * f);
                }
            }
        __syncthreads();
        const bool done = starts && ends;
        float *rec = a.part + ((int64_t)blockIdx.x * 2 + (starts ? 1 : 0)) * C::kRec;
        for (int i = tid; i < NC * (D / 2); i += 32 * kWarps) {
            const int col = i / (D / 2), d = i % (D / 2) * 2;
            float mt = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, s_m[w * NC + col]);
            float o0 = 0.f, o1 = 0.f, lt = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = s_m[w * NC + col];
                const float f = mw == -INFINITY ? 0.f : ex2(mw - mt);
                const float2 v = *(const float2 *)(s_o + (w * NC + col) * C::kOStride + d);
                // a warp without keys has l = 0 and o = 0
                lt = fmaf(f, s_l[w * NC + col], lt);
                o0 = fmaf(f, v.x, o0);
                o1 = fmaf(f, v.y, o1);
            }
            if (!done) {
                *(float2 *)(rec + col * D + d) = make_float2(o0, o1);
                if (d == 0) {
                    rec[NC * D + col] = mt;
                    rec[NC * D + NC + col] = lt;
                }
            } else if (c0 + col < s.ncol) {
                const int row = s.q0 + (c0 + col) / a.group, head = h * a.group + (c0 + col) % a.group;
                store_row(a, row, head * D + d, o0, o1, lt);
                if (d == 0 && a.lse)
                    a.lse[(int64_t)row * a.n_kv * a.group + head] =
                        lt == 0.f ? -INFINITY : (mt + log2f(lt)) * CUDART_LN2_F;
            }
        }
        __syncthreads();
        pos += take;
        off += take;
    }
    if (dead) {  // copies still in flight land before the shared memory goes
        int never = 0;
        for (; uses < fills; ++uses)
            tc::mbar_wait(&full[uses % kStages], (uses / kStages) & 1, a.timeout_cycles / 100 + 100000,
                          &never);
    }
}

// Joins the partial results of the item that CTA blockIdx.x of the split
// kernel began and did not finish, in CTA order.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps) moe_attn_join_kernel(MoeAttnArgs a, int ctas) {
    using C = Cfg<D, NT>;
    constexpr int NC = C::NC;
    __shared__ long long s_tot[kWarps], s_res[2];
    grid_dep_wait();
    grid_dep_launch();
    const long long total = total_work<NC>(a, false, s_tot);
    const long long per = piece_of(total, ctas, false);
    const long long cut = (blockIdx.x + 1) * per;  // where this CTA's piece ends
    if (cut >= total) return;
    int b;
    long long off;
    find_unit<NC>(a, false, cut - 1, s_tot, s_res, b, off);
    const Seq s = seq_of<NC>(a, b);
    const int item = (int)(off / s.tiles), u = (int)(off % s.tiles);
    if (u + 1 == s.tiles || u + 1 > per) return;  // ends here, or began before this CTA
    const int parts = 1 + (int)((s.tiles - (u + 1) + per - 1) / per);
    const int c0 = item / a.n_kv * NC, h = item % a.n_kv;
    const float *rec0 = a.part + ((int64_t)blockIdx.x * 2 + 1) * C::kRec;
    for (int i = threadIdx.x; i < NC * (D / 2); i += 32 * kWarps) {
        const int col = i / (D / 2), d = i % (D / 2) * 2;
        if (c0 + col >= s.ncol) continue;
        float mt = -INFINITY, lt = 0.f, o0 = 0.f, o1 = 0.f;
        for (int p = 0; p < parts; ++p) {
            const float *rec = p == 0 ? rec0 : a.part + ((int64_t)(blockIdx.x + p) * 2) * C::kRec;
            const float mp = rec[NC * D + col], lp = rec[NC * D + NC + col];
            const float2 v = *(const float2 *)(rec + col * D + d);
            const float mn = fmaxf(mt, mp);
            if (mp == -INFINITY) continue;  // no keys there
            const float f = ex2(mt - mn), w = ex2(mp - mn);
            lt = fmaf(lt, f, w * lp);
            o0 = fmaf(o0, f, w * v.x);
            o1 = fmaf(o1, f, w * v.y);
            mt = mn;
        }
        const int row = s.q0 + (c0 + col) / a.group, head = h * a.group + (c0 + col) % a.group;
        store_row(a, row, head * D + d, o0, o1, lt);
        if (d == 0 && a.lse)
            a.lse[(int64_t)row * a.n_kv * a.group + head] =
                lt == 0.f ? -INFINITY : (mt + log2f(lt)) * CUDART_LN2_F;
    }
}

// Two column tiles of 8 where a sequence may have more than 8 columns.
bool wide(int group, int max_q) { return (int64_t)group * max_q > 8; }

// A CTA takes whole items where each has at most a tile per warp.
bool whole_items(int max_kv) { return max_kv <= kWarps * kTile; }

template <int D, int NT>
cudaError_t launch(const MoeAttnArgs &a, int nsm, cudaStream_t st) {
    using C = Cfg<D, NT>;
    const bool whole = whole_items(a.b.max_kv);
    // no more CTAs than the bounds allow units
    const int64_t items = (int64_t)a.n_kv * ((int64_t)a.b.n_tokens * a.group / C::NC + a.b.n_seqs);
    const int64_t units = whole ? items : items * ((a.b.max_kv + kTile - 1) / kTile + 1) / kMinTiles + 1;
    const int ctas = (int)std::min<int64_t>(units, (int64_t)nsm * C::kCtasPerSm);
    cudaError_t err = cudaFuncSetAttribute(moe_attn_split_kernel<D, NT>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (err != cudaSuccess) return err;
    err = launch_pdl(moe_attn_split_kernel<D, NT>, dim3(ctas), dim3(32 * kWarps), C::kSmem, st, a, whole);
    if (err != cudaSuccess || whole) return err;
    return launch_pdl(moe_attn_join_kernel<D, NT>, dim3(ctas), dim3(32 * kWarps), 0, st, a, ctas);
}

}  // namespace

size_t moe_attn_ws_bytes(int head_dim, int group, int max_q, int max_kv, int nsm) {
    if (whole_items(max_kv)) return 0;
    const int nt = wide(group, max_q) ? 2 : 1, per_sm = nt == 2 ? 2 : 3;
    return (size_t)nsm * per_sm * 2 * (8 * nt * (head_dim + 2)) * sizeof(float);
}

cudaError_t moe_launch_attn(int head_dim, const MoeAttnArgs &a, int nsm, cudaStream_t st) {
    const bool w = wide(a.group, a.b.max_q);
    if (head_dim == 64) return w ? launch<64, 2>(a, nsm, st) : launch<64, 1>(a, nsm, st);
    return w ? launch<128, 2>(a, nsm, st) : launch<128, 1>(a, nsm, st);
}
