// Attention over the MXFP4 cache with many query rows per sequence: the same
// mathematics as the split kernel, on tcgen05 tensor cores.
//
// A CTA owns 256 columns (query rows x heads of one key/value head) of one
// sequence as two tiles A and B of 128, and runs over the keys in steps of 128,
// a step as two units of 64:
//   S_t = Q_t K^T        (128 x 64 x D, operands in shared memory, S in TMEM)
//   P_t = 2^(S_t - m)    (a thread per row: TMEM -> registers -> TMEM, fp16)
//   O_t += P_t V         (P from TMEM over S's columns, V from shared memory)
// Each tile has two S buffers: the products of the next unit run while the rows
// work on this one (one buffer of 128 keys instead, a step's products waiting
// for its softmax and the other way round: 361 us against 341 for 3 prompts of
// 2000 rows, 32 heads and up to 8000 keys). Warps 0-3 hold tile A's rows, 4-7
// tile B's, 8-13 turn the cache's codes into operands (each key and value once
// per CTA, i.e. once per 256 columns), 14 and 15 issue the tiles' MMAs. TMEM is
// full: S_A, S_B (two units each), O_A, O_B of 128 columns each.
//
// Operands are fp16: a code is exact, and its scale enters as 2^(e - R + 12)
// with R the largest key exponent (or, per block of 32 dimensions, the largest
// value exponent) that the CTA's rows can see, found in a pass over the scales
// before the loop; a block whose scale lies over 2^26 below the largest counts
// as 0. Queries as in the split kernel. Weights are rounded to fp16 as 2^5 p, so
// that a key loses 2^-30 of the maximum's weight at most (2^20 keys: half of the
// output's rounding); with 2^8 the maximum in use has to move more often (243 us
// against 230 for 3 prompts of 2000 rows). The maximum in use moves only when a
// unit's weights add up to more than 2^10 with it (they stay far inside fp16's
// range), so a unit is read once and no maximum of it is taken but for those
// few, which also rescale O (267 us for the same prompts with a maximum first,
// 254 without).
//
// Bound: 4 D flops per column and key on the tensor cores (the prompts above:
// 131 us of 235, their 256 columns and 128 keys in 2048 cycles); one exponential
// per column and key (32 a cycle and SM) is next. A step takes about 3500 cycles:
// a row warp's chain per unit (read, exponentials, write, two barriers) is longer
// than its products.
#include <algorithm>

#include "attn.cuh"

using namespace moe_attention;

namespace {

constexpr int kM = 128;          // rows of a tile (columns of the item)
constexpr int kCols = 2 * kM;    // columns of a CTA
constexpr int kN = 128;          // keys per step
constexpr int kU = kN / 2;       // keys per unit: of one S, one P
// warps 0-7 rows, 8-10 keys, 11-13 values, 14 and 15 MMA issue of tile A and B
// (one issuer's instructions take longer than the products: about 90 cycles
// each, against 64)
constexpr int kWarpsP = 16;
constexpr int kWarpK = 8, kWarpV = 11, kWarpMma = 14, kConv = 3;
constexpr int kThreadsP = 32 * kWarpsP;
constexpr int kInfo = 4;         // steps whose masks are kept
constexpr int kHead = 12;        // operands carry 2^12
constexpr int kUp = 5;           // weights carry 2^5
constexpr float kLag = 1024.f * (1 << kUp);  // what a unit's weights may add up to (64 x 2^5 at the row's maximum)

template <int D>
struct PCfg {
    static constexpr int NB = D / 32;
    static constexpr int kHalf = kM * 128;            // 128 rows of 64 elements
    static constexpr int kOp = kM * D * 2;            // an operand tile
    static constexpr int kSmemQ = 0, kSmemK = 2 * kOp, kSmemV = 4 * kOp;
    // + alignment; a second CTA on the SM would only wait for tensor memory
    static constexpr int kSmem = std::max(6 * kOp + 1024, 120 * 1024);
    static constexpr int kRec = kCols * (D + 2);      // floats of a partial result
};

struct StepInfo {
    union {
        struct {
            uint8_t any_gone[8], any_nan[8];  // by key or value warp
        };
        uint64_t any[2];  // the same, all at once
    };
    uint32_t gone[kConv][4];    // [warp][word]: tokens without a page in the cache
    uint32_t nan[kConv][4][4];  // [warp][block][word]: values that are NaN
};

// 32 consecutive TMEM columns of each lane; the registers hold them after
// tc::tmem_ld_wait().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
        "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {  // of the thread's own copies
    asm volatile("cp.async.wait_all;" ::: "memory");
}
// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// One lane of the warp, the same one every time; the compiler then knows that the
// branch has one thread and keeps an MMA's operands in uniform registers (297 us
// for the prompts below with lane 0 instead, 290 with this).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0u;
}
// D[tmem] (+)= A[tmem] x B[smem], fp16 operands, 16 K per instruction.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Descriptor of an MN-major operand, 128-byte swizzle: atoms of 64 elements
// (128 bytes) along MN x 8 along K; `mn` bytes between atoms along MN, 1024
// between atoms along K.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t mn) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(mn >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// kind::f16, fp16 operands, fp32 accumulator; bt: B is MN-major.
__device__ __forceinline__ uint32_t idesc_f16(int M, int N, bool bt) {
    return (1u << 4) | ((bt ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Factor pair 2^(e - R + 12) of a scale byte; 0 below fp16's normal range.
__device__ __forceinline__ uint32_t factor_of(uint32_t e, int R) {
    return (uint32_t)min(max((int)e - R + 15 + kHead, 0), 15 + kHead) * 0x04000400u;
}

// A warp's share of the codes of K or V (3 warps each, loads dealt in turn):
// each step into the operand buffer of its stage, the next step's codes on
// their way meanwhile. A lane takes one block of 32 dimensions of one token; 8
// tokens a quarter warp, so that codes are read in whole lines and written
// without bank conflicts. rmax: the exponent that the lane's block is taken
// against. (One code for both, which the six warps share in the instruction
// cache.)
template <int D, typename Wait>
__device__ __forceinline__ void convert(const MoeAttnArgs &a, bool v, int h, const int32_t *pages, int first,
                                        int n, int lo_all, int hi_all, int w, int rmax, uint8_t *ops,
                                        uint64_t *full, uint64_t *empty, StepInfo *info, const Wait &wait) {
    using C = PCfg<D>;
    constexpr int NB = C::NB, OCT = 4 / NB;  // octets of tokens that a load of the warp covers
    constexpr int LOADS = (16 / OCT + kConv - 1) / kConv;
    const int lane = threadIdx.x & 31, tl = lane & 7, k = (lane >> 3) % NB;
    const int in_page_mask = (1 << a.page_shift) - 1;
    const uint8_t *codes = v ? a.c.v_q : a.c.k_q, *scales = v ? a.c.v_s : a.c.k_s;
    uint4 cq[LOADS];
    uint32_t sb[LOADS], have = 0u;  // scale bytes; bit i: load i has its page
    int id[LOADS];                  // pages of the next step's loads
    const int row0 = 8 * (w * OCT + (lane >> 3) / NB) + tl;
    auto row_of = [&](int i) { return row0 + 8 * kConv * OCT * i; };  // token of load i within a step
    auto page_ids = [&](int j) {  // (-1: none; a step has kN tokens)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int tok = first + kN * j + row_of(i);
            id[i] = -1;
            if (j < n && row_of(i) < kN && tok < hi_all) id[i] = pages[tok >> a.page_shift];
        }
    };
    // this lane's block in the first octet of a page, and its scale
    const uint32_t page_scales = (uint32_t)a.n_kv * NB << a.page_shift;  // bytes of a page
    codes += ((uint64_t)h * NB << a.page_shift) * 16 + k * 128 + tl * 16;
    scales += (uint64_t)h * NB << a.page_shift;
    scales += v ? (tl & 6) * NB + 2 * k + (tl & 1) : tl * NB + k;
    auto load = [&](int j) {
        have = 0u;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            cq[i] = make_uint4(0u, 0u, 0u, 0u);
            sb[i] = 0u;
            // (nothing here may look at a loaded value: it would wait for it)
            if ((uint32_t)id[i] < (uint32_t)a.n_pages) {
                have |= 1u << i;
                const uint64_t at = (uint64_t)(uint32_t)id[i] * page_scales +
                                    (uint32_t)((first + kN * j + row_of(i)) & in_page_mask & ~7) * NB;
                cq[i] = *(const uint4 *)(codes + at * 16);
                sb[i] = scales[at];
            }
        }
    };
    uint8_t *const base = ops + (k >> 1) * C::kHalf + (row0 >> 3) * 1024 + tl * 128;
    int swz[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) swz[q] = ((4 * (k & 1) + q) ^ tl) << 4;
    page_ids(0);
    load(0);
    page_ids(1);
    for (int j = 0; j < n; ++j) {
        const int st = j & 1;
        if (!wait(&empty[st], ((j >> 1) & 1) ^ 1)) return;  // (a fresh barrier counts as passed)
        uint32_t odd = 0u;  // loads with tokens that every row leaves out, or NaN values: rare
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = row_of(i);
            if (r < kN) {
                // a NaN key makes its token's logits NaN (rows that do not see it
                // mask them); a NaN value counts as 0 here and reaches its rows at the end
                const bool nan = sb[i] == 255u;
                const uint32_t fac = nan ? (v ? 0u : 0x7E007E00u) : factor_of(sb[i], rmax);
                if (v ? nan && first + kN * j + r >= lo_all : !((have >> i) & 1u)) odd |= 1u << i;
                uint8_t *dst = base + st * C::kOp + i * (kConv * OCT * 1024);
                const uint32_t wd[4] = {cq[i].x, cq[i].y, cq[i].z, cq[i].w};
                uint32_t x[4][4];  // (all conversions first: 16 in flight)
#pragma unroll
                for (int q = 0; q < 4; ++q) codes_f16(wd[q], x[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int z = 0; z < 4; ++z) x[q][z] = mul_f16x2(x[q][z], fac);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *(uint4 *)(dst + swz[q]) = make_uint4(x[q][0], x[q][1], x[q][2], x[q][3]);
            }
        }
        StepInfo &f = info[j % kInfo];
        const bool any = __any_sync(kFull, odd != 0u);
        if (any) {
#pragma unroll 1
            for (int q = 0; q < 4 * NB; ++q) {  // word q % 4 (of block q / 4)
                uint32_t bits = 0u;
#pragma unroll
                for (int i = 0; i < LOADS; ++i)
                    if (((odd >> i) & 1u) && row_of(i) >> 5 == q % 4 && (!v || k == q / 4))
                        bits |= 1u << (row_of(i) & 31);
                bits = __reduce_or_sync(kFull, bits);
                if (lane == 0) {
                    if (v) f.nan[w][q / 4][q % 4] = bits;
                    else f.gone[w][q % 4] = bits;
                }
            }
        }
        if (lane == 0) (v ? f.any_nan : f.any_gone)[w] = any ? 1 : 0;
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&full[st]);
        load(j + 1);  // on its way over the wait
        page_ids(j + 2);
    }
}

// Column tiles of a sequence (p0 keys before its first row) whose last column
// sees L keys or more (its last ones), L >= 1.
__device__ __forceinline__ int tiles_from(int p0, int ncol, int cts, int group, int64_t L) {
    const int64_t c = (L - 1 - p0) * group;  // the first column that does
    return c <= 0 ? cts : c >= ncol ? 0 : cts - (int)c / kCols;
}

// Offset of a column's head row in the queries or the output, without a division
// per step of `by` columns.
struct Column {
    int64_t at, step, wrap;
    int head, group, rem;
    __device__ Column(int c, int by, int group_, int64_t stride, int width) : group(group_) {
        head = c % group;
        rem = by % group;
        at = c / group * stride + head * width;
        step = by / group * stride + rem * width;
        wrap = stride - group * width;
    }
    __device__ void next() {
        at += step;
        head += rem;
        if (head >= group) head -= group, at += wrap;
    }
};

// The r-th (sequence, column tile): the longest first, so that the last CTAs to
// start are short. The order is by the whole steps of keys that a tile sees,
// found by a search (32 lengths at a time, a lane each); for many sequences (whose
// CTAs are many) by column tile alone, or, where that would number too many tiles
// that do not exist (tiles_max 0), by sequence. False if there are fewer.
// Warp-collective.
__device__ __forceinline__ bool item_of(const MoeAttnArgs &a, int tiles_max, int r, int &b, int &ct) {
    const int lane = threadIdx.x & 31, B = a.b.n_seqs;
    if (B > 32 && tiles_max == 0) {
        for (int b0 = 0; b0 < B; b0 += 32) {
            const int cts = b0 + lane < B ? seq_of<kCols>(a, b0 + lane).cts : 0;
            int at = cts;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(kFull, at, off);
                if (lane >= off) at += o;
            }
            const uint32_t m = __ballot_sync(kFull, at > r);
            if (m != 0u) {
                b = b0 + __ffs(m) - 1;
                ct = __shfl_sync(kFull, at, b - b0) - 1 - r;  // the last tile first
                return true;
            }
            r -= __shfl_sync(kFull, at, 31);
        }
        return false;
    }
    if (B > 32) {
        b = r % B;
        ct = tiles_max - 1 - r / B;
        return ct >= 0 && ct * (int64_t)kCols < seq_of<kCols>(a, b).ncol;
    }
    Seq s = {};
    if (lane < B) s = seq_of<kCols>(a, lane);
    const int p0 = s.kv - s.nq;
    // the largest L with more than r tiles of L steps or more (0: any tile)
    int L = 0, end = a.b.max_kv / kN + 1;
    while (end - L > 1) {
        const int step = (end - L + 31) / 32;
        const int t = min(L + (lane + 1) * step, end);
        int count = 0;
#pragma unroll 4
        for (int i = 0; i < B; ++i)
            count += tiles_from(__shfl_sync(kFull, p0, i), __shfl_sync(kFull, s.ncol, i),
                                __shfl_sync(kFull, s.cts, i), a.group, (int64_t)kN * t);
        L += step * __popc(__ballot_sync(kFull, t < end && count > r));
        end = min(end, L + step);
    }
    // those of L steps, in order of sequence and tile, behind the longer ones
    const int more = lane < B ? tiles_from(p0, s.ncol, s.cts, a.group, (int64_t)kN * (L + 1)) : 0;
    const int from = lane < B ? (L == 0 ? s.cts : tiles_from(p0, s.ncol, s.cts, a.group, (int64_t)kN * L)) : 0;
    int skip = r - (int)__reduce_add_sync(kFull, (unsigned)more), at = from - more;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(kFull, at, off);
        if (lane >= off) at += o;
    }
    const uint32_t m = __ballot_sync(kFull, at > skip);
    if (m == 0u) return false;
    b = __ffs(m) - 1;
    skip -= __shfl_sync(kFull, at - (from - more), b);
    ct = __shfl_sync(kFull, s.cts - from, b) + skip;
    return true;
}

template <int D>
__global__ void __launch_bounds__(kThreadsP, 1)
    moe_attn_prefill_kernel(MoeAttnArgs a, int tiles_max, int splits) {
    using C = PCfg<D>;
    constexpr int NB = C::NB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2][2],
        p_full[2][2], o_part[2], o_full[2], q_full[2], drain[2];
    __shared__ StepInfo info[kInfo];
    __shared__ int s_rk, s_rv[NB], s_abort;
    __shared__ uint32_t s_tmem, s_bad[8];  // s_bad: rows of each row warp with a query that is not finite
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

    grid_dep_wait();
    grid_dep_launch();
    const int split = blockIdx.x % splits, blk = blockIdx.x / splits, h = blk % a.n_kv;
    int b, ct;
    if (!item_of(a, tiles_max, blk / a.n_kv, b, ct)) return;
    const Seq s = seq_of<kCols>(a, b);
    const int c0 = ct * kCols;
    const int G = a.group, p0 = s.kv - s.nq;
    const int i0 = c0 / G, i1 = (min(c0 + kCols, s.ncol) - 1) / G;
    const bool two = c0 + kM < s.ncol;  // tile B has columns
    const int hi_all = p0 + i1 + 1, W = a.b.window;
    const int lo_all = W > 0 ? max(0, p0 + i0 + 1 - W) : 0;
    const int begin = lo_all / 16 * 16;
    const int steps = hi_all > begin ? (hi_all - begin + kN - 1) / kN : 0;
    // (under 2^24 steps; splits that are at most the SMs)
    const int j0 = (int)((uint32_t)steps * split / splits), j1 = (int)((uint32_t)steps * (split + 1) / splits);
    const int n = j1 - j0, first = begin + kN * j0;
    const int32_t *pages = a.b.page_table + (int64_t)b * a.b.table_stride;
    const int in_page_mask = (1 << a.page_shift) - 1;

    if (tid == 32 * kWarpK) {  // (a warp without queries to fetch first)
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&k_full[i], kConv);
            tc::mbar_init(&k_empty[i], two ? 2 : 1);
            tc::mbar_init(&v_full[i], kConv);
            tc::mbar_init(&v_empty[i], two ? 2 : 1);
            tc::mbar_init(&drain[i], 1);
            tc::mbar_init(&s_full[i][0], 2);
            tc::mbar_init(&s_full[i][1], 1);
            tc::mbar_init(&q_full[i], 4);
            tc::mbar_init(&o_part[i], 1);
            tc::mbar_init(&o_full[i], 2);
            for (int k = 0; k < 2; ++k) tc::mbar_init(&p_full[i][k], 4);
        }
        for (int i = 0; i < kInfo; ++i) info[i].any[0] = info[i].any[1] = 0u;
        tc::fence_mbar_init();
        s_abort = 0;
        s_rk = 0;
        for (int k = 0; k < NB; ++k) s_rv[k] = 0;
    }
    if (wid == kWarpMma) {
        tc::tmem_alloc(&s_tmem, 512);
        tc::tmem_relinquish();
    }
    // --- queries: each row warp's 32 rows in whole lines into the operand's place,
    // while the scales are read
    constexpr int LPR = D / 8, ROWS = 32 / LPR;  // lanes of a row of 16-byte chunks, rows of a warp's pass
    const int chunk = lane % LPR;
    auto q_at = [&](int r, int ch) {
        return smem + C::kSmemQ + (r >> 7) * C::kOp + ((r & (kM - 1)) >> 3) * 1024 + (r & 7) * 128 +
               (ch >> 3) * C::kHalf + (((ch & 7) ^ (r & 7)) << 4);
    };
    const int scale_end = min(hi_all, first + kN * n);
    const int scale_page = first + 16 * tid < scale_end ? pages[(first + 16 * tid) >> a.page_shift] : -1;
    if (wid < 8) {
        const int r0 = tid & ~31;
        Column col(c0 + r0 + lane / LPR, ROWS, G, a.q_stride, D);
        const uint16_t *src = a.q + s.q0 * a.q_stride + h * G * D + 8 * chunk;
#pragma unroll 4
        for (int r = r0 + lane / LPR; r < r0 + 32; r += ROWS, col.next()) {
            if (c0 + r < s.ncol)
                cp_async16(q_at(r, chunk), src + col.at);
            else
                *(uint4 *)q_at(r, chunk) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __syncthreads();
    // --- the largest exponents that a row can see: 16 tokens (of one page) a thread
    {
        constexpr int WORDS = 4 * NB;  // of 16 tokens
        // maxima of e + 1 (0: NaN, or not seen) in 16 bits; V: [0] of the even
        // tokens (blocks 0, 1 and 2, 3), [1] of the odd ones
        uint32_t mk = 0u, mv[2][2] = {};
        int id = scale_page;
        for (int tok = first + 16 * tid; tok < scale_end; tok += 16 * kThreadsP) {
            if (tok >= first + 16 * kThreadsP) id = pages[tok >> a.page_shift];
            if (id < 0 || id >= a.n_pages) {
                moe_flag(a.status, MOE_ERR_BAD_INDEX);
                continue;
            }
            const int64_t row = (((int64_t)id * a.n_kv + h) << a.page_shift) + (tok & in_page_mask);
            uint32_t ks[WORDS], vs[WORDS];
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                *(uint4 *)(ks + i) = *(const uint4 *)(a.c.k_s + row * NB + 4 * i);
                *(uint4 *)(vs + i) = *(const uint4 *)(a.c.v_s + row * NB + 4 * i);
            }
            // bit i: token i is seen
            const int above = min(hi_all - tok, 16), below = max(lo_all - tok, 0);
            const uint32_t see = below >= 16 ? 0u : ((1u << above) - 1u) & ~((1u << below) - 1u);
            auto next16 = [](uint32_t w) { return (w & 0x00FF00FFu) + 0x00010001u & 0x00FF00FFu; };
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const int t0 = NB == 4 ? i & ~1 : 2 * i;  // the word's tokens: K t0 (and, NB 2, t0 + 1)
                const uint32_t s0 = (see >> t0) & 1u ? kFull : 0u, s1 = (see >> (t0 + 1)) & 1u ? kFull : 0u;
                const uint32_t k0 = next16(ks[i]), k1 = next16(ks[i] >> 8);
                if constexpr (NB == 4)
                    mk = __vmaxu2(mk, __vmaxu2(k0, k1) & (i & 1 ? s1 : s0));
                else
                    mk = __vmaxu2(mk, __vmaxu2(k0, k1) & ((s0 & 0xFFFFu) | (s1 & 0xFFFF0000u)));
                uint32_t(&m)[2] = mv[NB == 4 ? i & 1 : 0];
                m[0] = __vmaxu2(m[0], next16(vs[i]) & s0);
                m[1] = __vmaxu2(m[1], next16(vs[i] >> 8) & s1);
            }
        }
        mk = __reduce_max_sync(kFull, max(mk & 0xFFFFu, mk >> 16));
        if (lane == 0 && mk > 0u) atomicMax(&s_rk, (int)mk - 1);
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const uint32_t m = __vmaxu2(mv[k >> 1][0], mv[k >> 1][1]);
            const uint32_t v = __reduce_max_sync(kFull, k & 1 ? m >> 16 : m & 0xFFFFu);
            if (lane == 0 && v > 0u) atomicMax(&s_rv[k], (int)v - 1);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;
    const long long limit = a.timeout_cycles;
    // a bounded wait of a whole warp; false: give up
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        const bool ok = tc::mbar_wait_sleep(bar, parity & 1u, limit, &s_abort);
        if (__all_sync(kFull, ok)) return true;
        if (lane == 0) {
            moe_flag(a.status, MOE_ERR_DEVICE_TIMEOUT);
            *(volatile int *)&s_abort = 1;
        }
        return false;
    };

    if (wid < 8) {
        // ------------------------------------------------ softmax: a thread per row
        const int t = wid >> 2;
        const int c = c0 + tid;
        if (t == 0 || two) {
            // --- queries: fp16 with one power of two per row
            cp_async_wait();
            __syncwarp();
            uint32_t big = 0u;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint4 w = *(const uint4 *)q_at(tid, i);
                big = __vmaxu2(big, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                             __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
            }
            big = max(big & 0xFFFFu, big >> 16);
            // an infinity or NaN: the row goes through as zeros, so that keys that it does not
            // see stay out of it, and becomes NaN at the end if it saw any
            const bool bad = big >= 0x7F80u;
            const uint32_t bad_rows = __ballot_sync(kFull, bad);
            if (lane == 0) s_bad[wid] = bad_rows;  // (read behind the __syncwarp below)
            const int sh = min(141 - (int)(big >> 7), 127);
            // a negative scale's sign goes into the queries, so that the largest
            // product is the largest logit
            const float up = copysignf(pow2(sh), a.b.scale);
            // back from that power, |scale| log2(e)
            const float mul = bad ? 0.f : pow2(-sh) * (fabsf(a.b.scale) * CUDART_L2E_F);
            const uint32_t keep = bad ? 0u : kFull;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                uint4 *const at = (uint4 *)q_at(tid, i);
                uint32_t w[4] = {at->x, at->y, at->z, at->w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = pack_f16(__uint_as_float((w[k] & keep) << 16) * up,
                                    __uint_as_float(w[k] & keep & 0xFFFF0000u) * up);
                *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&q_full[t]);
            const uint32_t lanes = (uint32_t)(32 * (wid & 3)) << 16;
            const uint32_t sp = tmem + lanes + 128 * t, op = tmem + lanes + 256 + 128 * t;
            const int it0 = (c0 + kM * t) / G, it1 = (min(c0 + kM * (t + 1), s.ncol) - 1) / G;
            const int hi_min = p0 + it0 + 1, lo_max = W > 0 ? max(0, p0 + it1 + 1 - W) : 0;
            const int hi = c < s.ncol ? p0 + c / G + 1 : 0x7FFFFFFF;
            const int lo = c < s.ncol && W > 0 ? hi - W : 0;
            // logits: S x mul x 2^(R - 127 - 12); not 0, for masked columns are -inf
            float mr = mul * exp2f((float)(s_rk - 127 - kHead));
            if (mr == 0.f) mr = 1.17549435e-38f;
            // m: the maximum in use, less kUp; l is summed with its rounding errors in lc, so that
            // the weights of a long context count beside one that is far above them
            float m = -INFINITY, l = 0.f, lc = 0.f;
            // tokens tok0 + 32 q .. + 31 that the row sees
            auto seen = [&](int tok0, int q) {
                const int above = min(max(hi - (tok0 + 32 * q), 0), 32);
                const int below = min(max(lo - (tok0 + 32 * q), 0), 32);
                const uint32_t up = above == 32 ? kFull : (1u << above) - 1u;
                const uint32_t dn = below == 32 ? kFull : (1u << below) - 1u;
                return up & ~dn;
            };
            // blocks in which the row sees a NaN value in step j (read once PV(j)
            // was issued, so behind the value warps' masks)
            auto nan_seen = [&](int j) {
                const StepInfo &f = info[j % kInfo];
                uint32_t r = 0u;
                if (f.any[1] != 0u)
                    for (int w = 0; w < kConv; ++w)
                        if (f.any_nan[w])
                            for (int q = 0; q < 4; ++q)
                                for (int k = 0; k < NB; ++k)
                                    if (seen(first + kN * j, q) & f.nan[w][k][q]) r |= 1u << k;
                return r;
            };
            uint32_t nan_blocks = 0u;
            bool ok = true;
            uint32_t x[kU];
            bool there = false;  // the first half of the unit's logits is in x
            for (int u = 0; u < 2 * n; ++u) {
                const int j = u >> 1, side = u & 1;
                if (!there) {
                    if (!wait(&s_full[t][side], j)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    tmem_ld32(sp + kU * side, x);
                    tmem_ld32(sp + kU * side + 32, x + 32);
                    tc::tmem_ld_wait();  // (in the block of the loads: nothing may touch their registers before)
                } else {
                    tmem_ld32(sp + kU * side + 32, x + 32);
                    tc::tmem_ld_wait();
                }
                const StepInfo &f = info[j % kInfo];
                const int tok0 = first + kU * u;
                if (side == 0 && j > 0) nan_blocks |= nan_seen(j - 1);
                const bool gone = f.any[0] != 0u, some = tok0 + kU > hi_min || tok0 < lo_max || gone;
                // columns 32 q .. that the row does not see to -inf (few units have any)
                auto mask = [&](int q, uint32_t *y) {
                    uint32_t see = seen(tok0, q);
                    if (gone)
                        for (int w = 0; w < kConv; ++w)
                            if (f.any_gone[w]) see &= ~f.gone[w][kU / 32 * side + q];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((see >> i) & 1u)) y[i] = 0xFF800000u;
                };
                // weights of 32 logits into half as many registers; their sum
                auto weights = [&](const uint32_t *y, float ms, uint32_t *p) {
                    const uint64_t mr2 = pair(mr, mr), ms2 = pair(-ms, -ms);
                    uint64_t l2 = 0u;
#pragma unroll
                    for (int i = 15; i >= 0; --i) {
                        float y0, y1;
                        unpair(fma2(pair(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), mr2, ms2), y0, y1);
                        y0 = ex2(y0);
                        y1 = ex2(y1);
                        l2 = add2(l2, pair(y0, y1));
                        p[i] = pack_f16(y0, y1);
                    }
                    float l0, l1;
                    unpair(l2, l0, l1);
                    return l0 + l1;
                };
                if (some)
#pragma unroll
                    for (int q = 0; q < kU / 32; ++q) mask(q, x + 32 * q);
                const float ms = m == -INFINITY ? 0.f : m;
                uint32_t p[32];
                float sum = weights(x + 32, ms, p + 16) + weights(x, ms, p);
                if (!__any_sync(kFull, m == -INFINITY || !(sum <= kLag))) {
                    tmem_st32(sp + kU * side, p);
                } else {
                    // a row without a maximum yet, or one whose weights add up to too much:
                    // the unit goes again, with the rows' largest logits as the maximum
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int q = 0; q < kU / 32; ++q) {
                        uint32_t y[32];
                        tmem_ld32(sp + kU * side + 32 * q, y);
                        tc::tmem_ld_wait();
                        if (some) mask(q, y);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) mx = max3(mx, __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
                    }
                    const float top = mx * mr - (float)kUp;
                    const bool rise = top > m;
                    const float fac = rise && m > -INFINITY ? ex2(m - top) : 1.f;
                    if (u > 0) {  // O holds the units before, once S of unit u + 1, issued behind them, is there
                        if (!(u + 1 < 2 * n ? wait(&s_full[t][side ^ 1], (u + 1) >> 1) : wait(&o_part[t], 0))) {
                            ok = false;
                            break;
                        }
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t y[32];
                            tmem_ld32(op + 32 * q, y);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * fac);
                            tmem_st32(op + 32 * q, y);
                        }
                    }
                    if (rise) {
                        l *= fac;
                        lc *= fac;
                        m = top;
                    }
                    sum = 0.f;
#pragma unroll 1
                    for (int q = 0; q < kU / 32; ++q) {
                        uint32_t y[32];
                        tmem_ld32(sp + kU * side + 32 * q, y);
                        tc::tmem_ld_wait();
                        if (some) mask(q, y);
                        sum += weights(y, m == -INFINITY ? 0.f : m, p);
                        tmem_st16(sp + kU * side + 16 * q, p);
                    }
                }
                add_to(l, lc, sum);
                // half of the next unit's logits, if there, over the wait for the weights' store
                there = u + 1 < 2 * n &&
                        __all_sync(kFull, tc::mbar_try_wait(&s_full[t][side ^ 1], ((u + 1) >> 1) & 1));
                auto give = [&] {
                    tmem_st_wait();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&p_full[t][side]);
                };
                if (there) {
                    tc::tc_fence_after();
                    tmem_ld32(sp + kU * (side ^ 1), x);
                    give();
                    tc::tmem_ld_wait();
                } else {
                    give();
                }
            }
            // ------------------------------------------------ output
            // (without keys nothing else says that all four warps are done with the tile's
            // queries, which the output is staged over)
            if (ok) ok = wait(n > 0 ? &o_full[t] : &q_full[t], 0);
            if (ok) {
                tc::tc_fence_after();
                if (n > 0) nan_blocks |= nan_seen(n - 1);
                const bool live_row = c < s.ncol;
                const int row = s.q0 + c / G, head = h * G + c % G;
                float *rec = a.part + (int64_t)blockIdx.x * C::kRec + (int64_t)tid * (D + 2);
                l = (l - lc) * (1.f / (1 << kUp));
                if (((s_bad[wid] >> lane) & 1u) && l != 0.f) l = CUDART_NAN_F;
                const float r = l == 0.f ? 0.f : 1.f / l;  // (a row without keys: O is 0 too)
                // rows of the output meet in the tile's queries, which no product reads
                // any more, so that they leave in whole lines
                uint8_t *const own = smem + C::kSmemQ + wid * (32 * 2 * D);
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t x[32];
                    const float back = exp2f((float)(s_rv[q] - 127 - kHead - kUp));
                    if (n > 0) {
                        tmem_ld32(op + 32 * q, x);
                        tc::tmem_ld_wait();
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = n > 0 ? __float_as_uint(__uint_as_float(x[i]) * back) : 0u;
                    if ((nan_blocks >> q) & 1u) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = 0x7FFFFFFFu;
                    }
                    if (splits > 1) {
                        if (!live_row) continue;
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            *(float2 *)(rec + 32 * q + i) =
                                make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float y0 = __uint_as_float(x[8 * i + 2 * e]);
                                const float y1 = __uint_as_float(x[8 * i + 2 * e + 1]);
                                const __nv_bfloat162 v = __floats2bfloat162_rn(y0 * r, y1 * r);
                                w[e] = *reinterpret_cast<const uint32_t *>(&v);
                            }
                            *(uint4 *)(own + lane * (2 * D) + (((4 * q + i) ^ (lane & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (splits == 1) {
                    __syncwarp();
                    const int w0 = c0 + (tid & ~31);  // the warp's first column
                    Column col(w0 + lane / LPR, ROWS, G, a.out_stride, D);
                    uint16_t *dst = a.out + s.q0 * a.out_stride + h * G * D + 8 * chunk;
#pragma unroll 8
                    for (int i = lane / LPR; i < 32; i += ROWS, col.next())
                        if (w0 + i < s.ncol)
                            *(uint4 *)(dst + col.at) = *(const uint4 *)(own + i * (2 * D) + ((chunk ^ (i & 7)) << 4));
                }
                if (live_row && splits > 1) {
                    rec[D] = m;
                    rec[D + 1] = l;
                } else if (live_row && a.lse) {
                    a.lse[(int64_t)row * a.n_kv * G + head] =
                        l == 0.f ? -INFINITY : (m + (log2f(l) + kUp)) * CUDART_LN2_F;
                }
            }
            tc::tc_fence_before();
        }
    } else if (wid < kWarpMma) {
        // ------------------------------------------------ codes to operands
        const bool v = wid >= kWarpV;
        convert<D>(a, v, h, pages, first, n, lo_all, hi_all, wid - (v ? kWarpV : kWarpK),
                   v ? s_rv[(lane >> 3) % NB] : s_rk, smem + (v ? C::kSmemV : C::kSmemK), v ? v_full : k_full,
                   v ? v_empty : k_empty, info, wait);
    } else {
        // ------------------------------------------------ MMA issue of a tile (one lane)
        const int t = __shfl_sync(kFull, wid, 0) - kWarpMma;  // (uniform, to the compiler too)
        const uint32_t idesc_s = idesc_f16(kM, kU, false), idesc_o = idesc_f16(kM, D, true);
        const uint32_t sb = tc::smem_u32(smem), tm = __shfl_sync(kFull, tmem, 0), ts = tm + 128 * t, to = tm + 256 + 128 * t;
        const uint64_t qd = tc::sdesc_sw128(sb + C::kSmemQ + t * C::kOp);
        bool ok = true;
        if (t == 0 || two) {
            ok = wait(&q_full[t], 0);
            // S of unit u = Q K^T (by one lane)
            auto issue_s = [&](int u) {
                const int j = u >> 1, st = j & 1, side = u & 1;
                const uint64_t bd = tc::sdesc_sw128(sb + C::kSmemK + st * C::kOp + side * (kU * 128));
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint64_t o = (uint64_t)(((i >> 2) * C::kHalf + (i & 3) * 32) >> 4);
                    tc::mma_bf16(ts + kU * side, qd + o, bd + o, idesc_s, i > 0);
                }
                tc::mma_commit(&s_full[t][side]);
                if (side == 1) tc::mma_commit(&k_empty[st]);
                // orders the masks that were seen behind k_full (of this step) and v_full
                // (of the one before) before the rows' reads
                if (side == 0) tc::mbar_arrive(&s_full[t][0]);
            };
            if (n > 0 && ok) ok = wait(&k_full[0], 0);
            if (n > 0 && ok) {
                tc::tc_fence_after();
                if (elect_one()) {
                    issue_s(0);
                    issue_s(1);
                }
                __syncwarp();
            }
            // (test hook: nothing signals this barrier)
            if (a.inject == MOE_INJECT_ATTN_STALL && t == 0 && n > 0 && ok) ok = wait(&drain[t], 0);
            for (int u = 0; u < 2 * n && ok; ++u) {  // O += P V of unit u, then S of unit u + 2 over its P
                const int j = u >> 1, st = j & 1, side = u & 1;
                const bool more = j + 1 < n;
                // (the weights last: what they wait for is then issued without a pause)
                if (side == 0) ok = wait(&v_full[st], j >> 1) && (!more || wait(&k_full[st ^ 1], (j + 1) >> 1));
                ok = ok && wait(&p_full[t][side], j);
                if (!ok) break;
                tc::tc_fence_after();
                const uint64_t bd = sdesc_mn(sb + C::kSmemV + st * C::kOp, C::kHalf);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < kU / 16; ++i)
                        mma_f16_ts(to, ts + kU * side + 8 * i, bd + (uint64_t)((kU / 16 * side + i) * 2048 >> 4),
                                   idesc_o, (u > 0 || i > 0) ? 1u : 0u);
                    if (side == 1) tc::mma_commit(&v_empty[st]);
                    if (u == 2 * n - 2) tc::mma_commit(&o_part[t]);
                    if (u == 2 * n - 1) {
                        tc::mma_commit(&o_full[t]);
                        tc::mbar_arrive(&o_full[t]);  // (as above)
                    }
                    if (more) issue_s(u + 2);
                }
                __syncwarp();
            }
            // MMAs in flight end before TMEM goes, also where the rows give up on the last ones
            if (n > 0 && ok) ok = wait(&o_full[t], 0);
            if (!ok && elect_one()) tc::drain_mmas(&drain[t], limit);
        }
        __syncwarp();
    }
    __syncthreads();
    if (wid == kWarpMma) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Joins the splits of every column, in order: a warp per column.
template <int D>
__global__ void __launch_bounds__(256) moe_attn_prefill_join_kernel(MoeAttnArgs a, int tiles_max, int splits) {
    using C = PCfg<D>;
    grid_dep_wait();
    grid_dep_launch();
    const int col = (blockIdx.x % (kCols / 8)) * 8 + (threadIdx.x >> 5), blk = blockIdx.x / (kCols / 8);
    const int lane = threadIdx.x & 31, h = blk % a.n_kv;
    int b, ct;
    if (!item_of(a, tiles_max, blk / a.n_kv, b, ct)) return;
    const Seq s = seq_of<kCols>(a, b);
    const int c = ct * kCols + col;
    if (c >= s.ncol) return;
    const float *rec = a.part + (int64_t)blk * splits * C::kRec + (int64_t)col * (D + 2);
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
    for (int p = 0; p < splits; ++p) m = fmaxf(m, rec[p * C::kRec + D]);
#pragma unroll 4
    for (int p = 0; p < splits; ++p) {
        const float *r = rec + p * C::kRec;
        const float f = r[D] == -INFINITY && r[D + 1] == 0.f ? 0.f : ex2(r[D] - m);
        l = fmaf(f, r[D + 1], l);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const float2 v = *(const float2 *)(r + 64 * i + 2 * lane);
            // (a part without keys holds zeros)
            o[2 * i] = fmaf(f, v.x, o[2 * i]);
            o[2 * i + 1] = fmaf(f, v.y, o[2 * i + 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
        store_out(a, s.q0 + c / a.group, h * a.group + c % a.group, D, 64 * i + 2 * lane, o[2 * i], o[2 * i + 1], m, l, kUp);
}

constexpr int kSplitKeys = 4 * kN;   // keys of a split at least
constexpr int kOneReadCols = 16;     // columns for which the split kernel reads the cache once

struct Shape {
    int tiles_max, splits;  // (see item_of; column tiles of the longest sequence)
    int64_t ctas;
};

Shape shape_of(const moe_attn_batch &q, int n_kv, int group, int nsm) {
    Shape r;
    const int64_t tiles_max = ((int64_t)q.max_q * group + kCols - 1) / kCols;
    // column tiles of all sequences, by either bound
    const int64_t grid = tiles_max * q.n_seqs, most = (int64_t)q.n_tokens * group / kCols + q.n_seqs;
    // 8 prompts of 2000 rows among 248 single rows, 64 / 8 heads: grid is 16128 and
    // most 763 tiles a key/value head, and a CTA without a tile costs its start: 2.75
    // and 1.95 ms
    const bool ragged = q.n_seqs > 32 && grid > 4 * most;
    r.tiles_max = ragged ? 0 : (int)tiles_max;
    const int64_t items = (q.n_seqs > 32 && !ragged ? grid : std::min(grid, most)) * n_kv;
    // few items: split the keys so that the SMs are all used
    r.splits = (int)std::max<int64_t>(1, std::min<int64_t>(nsm / std::max<int64_t>(items, 1),
                                                           std::max(1, q.max_kv / kSplitKeys)));
    r.ctas = items * r.splits;
    return r;
}

template <int D>
cudaError_t launch(const MoeAttnArgs &a, int nsm, cudaStream_t st) {
    using C = PCfg<D>;
    const Shape g = shape_of(a.b, a.n_kv, a.group, nsm);
    const cudaError_t err = launch_pdl_ready(moe_attn_prefill_kernel<D>, dim3((unsigned)g.ctas), dim3(kThreadsP), C::kSmem, st, a,
                     g.tiles_max, g.splits);
    if (err != cudaSuccess || g.splits == 1) return err;
    return launch_pdl_ready(moe_attn_prefill_join_kernel<D>, dim3((unsigned)(g.ctas / g.splits * (kCols / 8))),
                      dim3(256), 0, st, a, g.tiles_max, g.splits);
}

template <int D>
cudaError_t setup() {
    const cudaError_t err = set_kernel((const void *)moe_attn_prefill_kernel<D>, PCfg<D>::kSmem);
    return err != cudaSuccess ? err : set_kernel((const void *)moe_attn_prefill_join_kernel<D>);
}

}  // namespace

cudaError_t moe_attn_prefill_setup() {
    const cudaError_t err = setup<64>();
    return err != cudaSuccess ? err : setup<128>();
}

bool moe_attn_prefill_fits(int n_seqs, int n_kv, int group, int max_q, int max_kv) {
    // The split kernel reads the cache once for every 16 columns, this one once for
    // 256, but its CTAs take a while to start. 16 sequences of 4000 keys, 8
    // key/value heads: 46 us there and 63 here with 16 columns, 76 and 63 with 24,
    // 139 and 64 with 64; one such sequence: 18 and 25 with 32 columns, 22 and 26
    // with 64 (from there on always here: longer batches gain), 29 and 29 with 128.
    const int64_t cols = (int64_t)group * max_q;
    if (cols <= kOneReadCols) return false;
    if (cols < MOE_ATTN_PREFILL_COLS &&
        (double)cols * n_seqs * n_kv * max_kv < MOE_ATTN_PREFILL_LOGITS)
        return false;
    return true;
}

size_t moe_attn_prefill_ws_bytes(int head_dim, int group, int max_q, int max_kv, int nsm) {
    // a partial result per CTA where the keys are split: then there are nsm CTAs at most
    if ((int64_t)group * max_q <= kOneReadCols || max_kv < 2 * kSplitKeys) return 0;
    return (size_t)nsm * kCols * (head_dim + 2) * sizeof(float);
}

cudaError_t moe_launch_attn_prefill(int head_dim, const MoeAttnArgs &a, int nsm, cudaStream_t st) {
    return head_dim == 64 ? launch<64>(a, nsm, st) : launch<128>(a, nsm, st);
}
