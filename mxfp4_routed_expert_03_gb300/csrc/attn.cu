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
// 2^29 below the largest vanish). p itself is rounded to fp16 (11 bits) as
// 2^10 p, so that a warp's sum loses 2^-35 of the largest weight a key at most,
// and its factor is 2^(5 + e - R).
// Queries are put into fp16 with one power of two per row, exact for elements
// within 2^-29 of the row's largest.
//
// Split. Tokens go in tiles of 32. The tiles of all (sequence, column tile,
// head) items form one line, with a fixed cost before each item's, that is cut
// into equal pieces, one per CTA, so any mix of lengths is balanced; few items
// are cut into equal parts instead, so that no CTA meets two of them. A CTA's fifth warp walks the piece ahead of the others and
// fills a ring of stages with bulk copies, across item ends; four warps take a
// tile of each stage, each with its own m, l, o, and merge at an item's end;
// items cut between CTAs leave partial results that a second kernel joins in
// a fixed order.
#include <limits.h>

#include <algorithm>

#include "attn.cuh"

using namespace moe_attention;

namespace {

constexpr int kWarps = 4;              // that compute, a tile each; one more fills the ring
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 3;
constexpr int kMinTiles = kWarps;      // of a piece
constexpr int kUp = 10;                // weights carry 2^10 (see above)
// An item's start and end in tiles, at 8, 12 and 16: 64 ragged sequences to 8192 keys 52.2,
// 48.4 and 48.0 us, 16 to 4000 keys 22.3, 21.3 and 21.4, 24 of 5 rows 19.6, 19.7 and 20.7, 32 equal ones
// of 2000 keys 31.8, 32.1 and 32.7.
constexpr int kItemCost = 12;

template <int D, int NT>
struct Cfg {
    static constexpr int NB = D / 32;             // blocks of a head row
    static constexpr int NC = 8 * NT;             // columns of a tile
    static constexpr int kCode = kTile * D / 2;   // bytes of a tile's K (or V) codes
    static constexpr int kScale = kTile * NB;
    static constexpr int kTileBytes = 2 * (kCode + kScale);
    static constexpr int kStage = kWarps * kTileBytes;
    static constexpr int kOStride = D + 4;
    static constexpr int kSmemO = kStages * kStage;
    static constexpr int kSmem = kSmemO + kWarps * NC * kOStride * 4;
    static constexpr int kCtasPerSm = NT == 1 ? 3 : 2;
    static constexpr int kRec = NC * (D + 2);     // floats of a partial result: o, m, l
    static constexpr int kHead = 8;               // words of a CTA's header: see Cut
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
// The same from a zero accumulator.
__device__ __forceinline__ void mma_f16_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void bulk_g2s(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            tc::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
        : "memory");
}

// The factor 2^(15 - kUp + y) of a value scale 2^y times the largest (y <= 0; more counts as
// 0) in fp16: subnormal below 2^-14, 0 below 2^-24.
__device__ __forceinline__ uint32_t factor(int y) {
    const int e = 15 - kUp + min(y, 0);
    return e >= -14 ? (uint32_t)(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
}
// R of a stored (15 - R) x 65537.
__device__ __forceinline__ int max_exp(uint32_t r15) { return 15 - (int)r15 / 65537; }

// ------------------------------------------------------------------ schedule
// How the items are dealt to the CTAs.
enum Deal {
    DEAL_WHOLE,  // whole items, a contiguous run of them each (short sequences)
    DEAL_PARTS,  // few items: each cut into the same number of parts, a CTA per part
    DEAL_LINE    // all items' tiles, and kItemCost units before each item's, on one
                 // line that is cut into equal pieces
};

// A sequence's share: items and units of the line.
struct Share {
    long long items, units;
};
template <int NC>
__device__ __forceinline__ Share share_of(const MoeAttnArgs &a, int b, int &tiles) {
    const Seq s = seq_of<NC>(a, b);
    Share r;
    r.items = (long long)s.cts * a.n_kv;
    r.units = r.items * (kItemCost + s.tiles);
    tiles = r.items > 0 ? s.tiles : 0;
    return r;
}

struct ScanSpace {
    Share tot[kWarps + 1];
    int tiles[kWarps + 1];
    long long res[2];
};

// Inclusive prefix over the block's threads, their sum, and the largest `tiles`.
__device__ __forceinline__ Share block_scan(Share v, int &tiles, ScanSpace &sp, Share &incl) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long i = __shfl_up_sync(kFull, incl.items, off), u = __shfl_up_sync(kFull, incl.units, off);
        if (lane >= off) incl.items += i, incl.units += u;
    }
    tiles = __reduce_max_sync(kFull, tiles);
    __syncthreads();
    if (lane == 31) sp.tot[wid] = incl, sp.tiles[wid] = tiles;
    __syncthreads();
    Share sum = {0, 0}, before = {0, 0};
#pragma unroll
    for (int w = 0; w <= kWarps; ++w) {
        if (w == wid) before = sum;
        sum.items += sp.tot[w].items;
        sum.units += sp.tot[w].units;
        tiles = max(tiles, sp.tiles[w]);
    }
    incl.items += before.items;
    incl.units += before.units;
    return sum;
}

// The whole batch's share and its longest item. `mine` and `incl` get the
// calling thread's sequence of the first round (the only one for up to kThreads
// sequences) and its inclusive prefix.
template <int NC>
__device__ Share total_share(const MoeAttnArgs &a, ScanSpace &sp, int &tiles, Share &mine, Share &incl) {
    Share sum = {0, 0};
    tiles = 0;
    for (int base = 0; base < a.b.n_seqs; base += kThreads) {
        const int b = base + threadIdx.x;
        Share v = {0, 0}, in;
        int t = 0;
        if (b < a.b.n_seqs) v = share_of<NC>(a, b, t);
        const Share r = block_scan(v, t, sp, in);
        sum.items += r.items;
        sum.units += r.units;
        tiles = max(tiles, t);
        if (base == 0) mine = v, incl = in;
    }
    return sum;
}

// The sequence that holds position `pos` (0 <= pos < total) of the items (or,
// `line`, of the units), and the position's offset in it.
template <int NC>
__device__ void find_seq(const MoeAttnArgs &a, bool line, long long pos, Share mine, Share incl, ScanSpace &sp,
                         int &seq, long long &off) {
    long long before = 0;
    for (int base = 0; base < a.b.n_seqs; base += kThreads) {
        const int b = base + threadIdx.x;
        long long sum = -1;  // (not needed when the first round is the only one)
        if (a.b.n_seqs > kThreads) {
            int t = 0;
            mine = {0, 0};
            if (b < a.b.n_seqs) mine = share_of<NC>(a, b, t);
            const Share r = block_scan(mine, t, sp, incl);
            sum = line ? r.units : r.items;
        }
        const long long n = line ? mine.units : mine.items, first = before + (line ? incl.units : incl.items) - n;
        if (pos >= first && pos < first + n) {
            sp.res[0] = b;
            sp.res[1] = pos - first;
        }
        if (pos < before + sum) break;  // block-uniform
        before += sum;
    }
    __syncthreads();
    seq = (int)sp.res[0];
    off = sp.res[1];
}

// Written by every CTA of the split kernel: the item that it began and did not
// finish (parts CTAs hold its pieces), parts = 0 if there is none.
struct Cut {
    int parts, q0, c0, ncol, head;
    int pad[3];
};

__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"r"(32 * kWarps) : "memory");
}

// ------------------------------------------------------------------ kernel
// A CTA's work, item by item.
struct Walk {
    int deal;
    long long pos, end;  // items or units still to take
    long long off;       // of the next one in its sequence
    int b;
    int part, parts;     // DEAL_PARTS: the CTA's part of its item
    long long per;       // DEAL_LINE: units of a piece
};

// One item (or part) of a CTA: a column tile and head of a sequence, token
// tiles [x_lo, x_hi) of which hold keys that some column sees.
struct Item {
    Seq s;
    int c0, h;
    int p0;                              // position of query row 0
    int hi_min, hi_max, lo_min, lo_max;  // key bounds over the columns
    int x_lo, x_hi;
    int parts;                           // CTAs that hold a part of the item, from the first on
    bool starts;                         // this is the first
    int b;
};

template <int NC>
__device__ __forceinline__ bool next_item(const MoeAttnArgs &a, Walk &w, Item &it) {
    while (w.pos < w.end) {
        it.s = seq_of<NC>(a, w.b);
        const Seq &s = it.s;
        const int units = w.deal == DEAL_LINE ? kItemCost + s.tiles : 1;
        if (w.off >= (long long)s.cts * a.n_kv * units) {  // past the sequence's last item
            ++w.b;
            w.off = 0;
            continue;
        }
        int item, tb = 0, te = s.tiles;
        it.starts = true;
        it.parts = 1;
        if (w.deal == DEAL_LINE) {
            item = (int)(w.off / units);
            const int u0 = (int)(w.off - (long long)item * units);
            const int take = (int)min((long long)(units - u0), w.end - w.pos);
            w.pos += take;
            w.off += take;
            tb = max(0, u0 - kItemCost);
            te = u0 + take - kItemCost;
            if (te <= tb) continue;  // the piece ends before the item's first tile
            it.starts = tb == 0;
            it.parts = 1 + (int)((units - u0 - take + w.per - 1) / w.per) + (it.starts ? 0 : 1);
        } else {
            item = (int)w.off;
            ++w.pos;
            ++w.off;
            if (w.deal == DEAL_PARTS) {
                it.parts = min(w.parts, s.tiles);
                if (w.part >= it.parts) continue;
                tb = (int)((long long)s.tiles * w.part / it.parts);
                te = (int)((long long)s.tiles * (w.part + 1) / it.parts);
                it.starts = w.part == 0;
            }
        }
        it.b = w.b;
        it.c0 = item / a.n_kv * NC;
        it.h = item % a.n_kv;
        const int i0 = it.c0 / a.group, i1 = (min(it.c0 + NC, s.ncol) - 1) / a.group;
        it.p0 = s.kv - s.nq;
        it.hi_max = it.p0 + i1 + 1;
        it.hi_min = it.p0 + i0 + 1;
        it.lo_min = a.b.window > 0 ? max(0, it.hi_min - a.b.window) : 0;
        it.lo_max = a.b.window > 0 ? max(0, it.hi_max - a.b.window) : 0;
        it.x_lo = max(tb, (it.lo_min - s.lo) / kTile);
        it.x_hi = it.hi_max <= s.lo ? it.x_lo
                                    : max(it.x_lo, min(te, (it.hi_max - s.lo + kTile - 1) / kTile));
        return true;
    }
    return false;
}

// The warp that fills the ring: for every item of the piece, stage by stage,
// K codes, V codes, K scales and V scales of 4 tiles. Lane = tile * 8 + array
// * 2 + page of the tile (two where pages hold 16 tokens).
template <int D, int NT>
__device__ __forceinline__ void fill_ring(const MoeAttnArgs &a, Walk walk, uint8_t *smem,
                                          uint64_t *full, uint64_t *empty, uint32_t (*valid)[kWarps],
                                          int *abort_flag) {
    using C = Cfg<D, NT>;
    const int lane = threadIdx.x & 31;
    const int tile = lane >> 3, which = (lane >> 1) & 3, part = lane & 1;
    const int parts = a.page_shift == 4 ? 2 : 1;
    const int unit = which < 2 ? C::NB * 16 : C::NB;  // bytes of a token
    const uint8_t *src0 = which == 0   ? a.c.k_q
                          : which == 1 ? a.c.v_q
                          : which == 2 ? a.c.k_s
                                       : a.c.v_s;
    uint8_t *const dst0 = smem + tile * C::kTileBytes +
                          (which < 2 ? which * C::kCode : 2 * C::kCode + (which - 2) * C::kScale) +
                          16 * part * unit;
    const uint32_t bytes = (uint32_t)(unit * kTile) / parts;
    int st = 0;
    uint32_t par = 1;  // of the empty barriers: a fresh one counts as passed
    int fills = 0;
    auto wait = [&](uint64_t *bar, uint32_t parity) {  // bounded; false: give up
        const bool ok = tc::mbar_wait_sleep(bar, parity, a.timeout_cycles, abort_flag);
        if (__all_sync(kFull, ok)) return true;
        if (lane == 0) {
            moe_flag(a.status, MOE_ERR_DEVICE_TIMEOUT);
            *(volatile int *)abort_flag = 1;
        }
        return false;
    };
    Item it;
    while (next_item<C::NC>(a, walk, it)) {
        const int32_t *pages = a.b.page_table + (int64_t)it.b * a.b.table_stride;
        // the item's queries, which the other warps load when they get there
        for (int i = lane; i < C::NC * (D / 64); i += 32) {
            const int c = it.c0 + i / (D / 64);
            if (c < it.s.ncol)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(
                    a.q + (int64_t)(it.s.q0 + c / a.group) * a.q_stride + (it.h * a.group + c % a.group) * D +
                    i % (D / 64) * 64));
        }
        // the page of this lane's tile of the stage at tile x (-2: not needed; the first
        // of a tile's two pages may lie wholly before the window)
        const int from = parts == 2 ? it.lo_min - 16 : INT_MIN;
        auto page_at = [&](int x) {
            const int tok = it.s.lo + kTile * (x + tile) + 16 * part;
            if (part >= parts || x + tile >= it.x_hi || tok >= it.hi_max || tok <= from) return -2;
            const int id = pages[tok >> a.page_shift];
            return id >= 0 && id < a.n_pages ? id : -1;
        };
        int id = page_at(it.x_lo);
        for (int x = it.x_lo; x < it.x_hi; x += kWarps) {
            if (id == -1) moe_flag(a.status, MOE_ERR_BAD_INDEX);
            const int next = page_at(x + kWarps);  // in flight over the wait
            if (!wait(&empty[st], par)) goto wind_down;
            const uint32_t have = __ballot_sync(kFull, which == 0 && id >= 0);
            if ((lane & 7) == 0) {
                const uint32_t two = have >> lane;  // bit 0: first page, bit 1: second
                valid[st][tile] = parts == 2 ? (two & 1u ? 0xFFFFu : 0u) | (two & 2u ? 0xFFFF0000u : 0u)
                                             : (two & 1u ? kFull : 0u);
            }
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive_expect_tx(&full[st], __popc(have) * (C::kTileBytes / parts));
            __syncwarp();
            if (id >= 0) {
                const int in_page = (it.s.lo + kTile * (x + tile) + 16 * part) & ((1 << a.page_shift) - 1);
                const int64_t row = (((int64_t)id * a.n_kv + it.h) << a.page_shift) + in_page;
                bulk_g2s(dst0 + st * C::kStage, src0 + row * unit, bytes, &full[st]);
            }
            id = next;
            ++fills;
            if (++st == kStages) st = 0, par ^= 1u;
            // (test hook: nothing signals this barrier)
            if (a.inject == MOE_INJECT_ATTN_STALL && !wait(&empty[kStages], 0u)) goto wind_down;
        }
    }
wind_down:  // copies in flight land before the shared memory goes, whether or not a warp waits for them
    int never = 0;
    for (int i = 0; i < kStages; ++i) {
        const int rounds = fills > i ? (fills - i + kStages - 1) / kStages : 0;
        if (rounds > 0)
            tc::mbar_wait(&full[i], (uint32_t)((rounds - 1) & 1), a.timeout_cycles / 100 + 100000, &never);
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtasPerSm)
    moe_attn_split_kernel(MoeAttnArgs a, bool whole) {
    using C = Cfg<D, NT>;
    constexpr int NB = C::NB, NC = C::NC;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ ScanSpace s_scan;
    __shared__ __align__(16) uint32_t s_scale[kWarps][kTile * NB + kTile / 2 * NB];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages + 1];  // (empty: one more for the test hook)
    __shared__ uint32_t valid[kStages][kWarps];
    __shared__ float s_m[kWarps * NC], s_l[kWarps * NC];
    __shared__ int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    float *s_o = (float *)(smem + C::kSmemO);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], kWarps);
        }
        tc::mbar_init(&empty[kStages], 1);
        s_abort = 0;
        tc::fence_mbar_init();
    }
    grid_dep_wait();
    grid_dep_launch();
    Share mine = {0, 0}, incl = {0, 0};
    int longest;
    const Share all = total_share<NC>(a, s_scan, longest, mine, incl);
    Cut *cut = (Cut *)a.part + blockIdx.x;
    float *const recs = a.part + (size_t)gridDim.x * C::kHead;
    if (tid == 0 && !whole) cut->parts = 0;
    if (all.items == 0) return;
    Walk walk;
    walk.part = 0;
    walk.parts = 1;
    walk.per = 1;
    // Parts of an item, if every CTA took one; at the finest. Equal parts where there
    // are four of an item or all it can have: one sequence of 777 keys 9.2 us (on the
    // line, where a CTA meets two items, 13.4), four of 5000 14.5 (15.7). Where parts are
    // long the line, which leaves no CTA idle, is 1 to 3 % faster: two of 100000 64.5
    // (63.2), two of 262143 146 (141).
    const int cap = (int)((long long)gridDim.x / all.items), fine = (longest + kMinTiles - 1) / kMinTiles;
    walk.deal = whole ? DEAL_WHOLE : cap >= min(fine, 4) ? DEAL_PARTS : DEAL_LINE;
    if (walk.deal == DEAL_WHOLE) {
        const long long per = (all.items + gridDim.x - 1) / gridDim.x;
        walk.pos = blockIdx.x * per;
        walk.end = min(all.items, walk.pos + per);
    } else if (walk.deal == DEAL_PARTS) {
        walk.parts = min(cap, fine);
        walk.pos = blockIdx.x / walk.parts;
        walk.part = blockIdx.x % walk.parts;
        walk.end = min(all.items, walk.pos + 1);
    } else {
        walk.per = max((all.units + gridDim.x - 1) / gridDim.x, (long long)(kItemCost + kMinTiles));
        walk.pos = blockIdx.x * walk.per;
        walk.end = min(all.units, walk.pos + walk.per);
    }
    if (walk.pos >= walk.end) return;
    find_seq<NC>(a, walk.deal == DEAL_LINE, walk.pos, mine, incl, s_scan, walk.b, walk.off);
    if (wid == kWarps) {
        fill_ring<D, NT>(a, walk, smem, full, empty, valid, &s_abort);
        return;
    }
    uint32_t *const kf = s_scale[wid], *const vf = kf + kTile * NB;  // scales of the warp's tile
    const int vpair = NB == 4 ? lane >> 1 : lane & 15, vhalf = NB == 4 ? lane & 1 : 0;
    const uint32_t lane_off = (lane & 8) * (NB * 16) + (lane >> 4) * 128 + (lane & 7) * 16;
    int use_st = 0;
    uint32_t use_par = 0;
    bool dead = false;  // a wait ran out
    Item it;
    while (next_item<NC>(a, walk, it)) {
        const Seq &s = it.s;
        const int c0 = it.c0, h = it.h, p0 = it.p0;

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

        // m: the running maximum less kUp; ms: the same as weights are taken against it, 0 while
        // there is none
        float o[NB][2][NT][4], m[NT][2], ms[NT][2], l[NT][2], lc[NT][2];  // (l: see add_to)
        // (15 - R) in both halves, as one product so that nothing carries between
        // them, of this lane's two blocks (see the scales below)
        uint32_t r15[2] = {15u * 65537u, 15u * 65537u};
#pragma unroll
        for (int k = 0; k < NB; ++k) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[k][hh][n][c] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, ms[n][0] = ms[n][1] = l[n][0] = l[n][1] = lc[n][0] = lc[n][1] = 0.f;

        for (int x = it.x_lo; x < it.x_hi && !dead; x += kWarps) {
            const int st = use_st;
            const uint32_t par = use_par;
            if (++use_st == kStages) use_st = 0, use_par ^= 1u;
            if (x + wid >= it.x_hi) {  // no tile of this stage for this warp
                if (lane == 0) tc::mbar_arrive(&empty[st]);
                continue;
            }
            const bool ok = tc::mbar_wait(&full[st], par, a.timeout_cycles, &s_abort);
            if (!__all_sync(kFull, ok)) {
                if (lane == 0) {
                    moe_flag(a.status, MOE_ERR_DEVICE_TIMEOUT);
                    *(volatile int *)&s_abort = 1;
                }
                dead = true;
                break;
            }
            const uint8_t *buf = smem + st * C::kStage + wid * C::kTileBytes;
            const uint32_t base = tc::smem_u32(buf);
            const int tok0 = s.lo + kTile * (x + wid);
            const uint32_t live = valid[st][wid];
            const bool edge = tok0 + kTile > it.hi_min || tok0 < it.lo_max || live != kFull;

            // --- scales, once for the warp. Keys: lane = token, 2^(byte - 127) of its
            // blocks in fp32; the lowest bit set makes 255 a NaN (and is a 2^-23
            // error otherwise), 2^-127 is a subnormal.
            {
                const uint8_t *ks = buf + 2 * C::kCode + lane * NB;
                const uint32_t w = NB == 4 ? *(const uint32_t *)ks : *(const uint16_t *)ks;
                uint32_t f[NB];
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    f[k] = (k == 0 ? w << 23 : k == 1 ? w << 15 : k == 2 ? w << 7 : w >> 1) & 0x7F800000u;
                    f[k] = f[k] == 0u ? 0x00400000u : f[k] | 1u;
                }
                if constexpr (NB == 4) *(uint4 *)(kf + 4 * lane) = make_uint4(f[0], f[1], f[2], f[3]);
                else *(uint2 *)(kf + 2 * lane) = make_uint2(f[0], f[1]);
            }
            // Values: lane = token pair and pair of blocks, factor(e - R) of both
            // tokens as an fp16 pair. e - R + 15 is in 0 .. 15 for all but few tiles.
            bool special = false;  // a scale that is NaN
            {
                const uint32_t w = *(const uint32_t *)(buf + 2 * C::kCode + C::kScale + vpair * (2 * NB) + 4 * vhalf);
                uint32_t e2[2] = {__byte_perm(w, 0u, 0x4140), __byte_perm(w, 0u, 0x4342)};
                if (edge) {  // tokens that no column sees must not move R (their weight is 0)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int i = 2 * vpair + e, tk = tok0 + i;
                        if (tk >= it.hi_max || tk < it.lo_min || !((live >> i) & 1u)) {
                            const uint32_t half = 0xFFFFu << (16 * e);
                            e2[0] = (e2[0] & ~half) | ((uint32_t)max_exp(r15[0]) << (16 * e));
                            e2[1] = (e2[1] & ~half) | ((uint32_t)max_exp(r15[1]) << (16 * e));
                        }
                    }
                }
                uint32_t d0 = e2[0] + r15[0], d1 = e2[1] + r15[1];
                if (__any_sync(kFull, ((d0 | d1) & 0xFFF0FFF0u) != 0u)) {
                    float back[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t old = (uint32_t)max_exp(r15[j]);
                        uint32_t top = old;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t y = (e2[j] >> (16 * e)) & 0xFFFFu;
                            if (y == 255u) special = true;
                            else top = max(top, y);
                        }
#pragma unroll
                        for (int off = NB / 2; off < 32; off <<= 1) top = max(top, __shfl_xor_sync(kFull, top, off));
                        back[j] = exp2f((float)((int)old - (int)top));
                        r15[j] = (15u - top) * 65537u;
                        const uint32_t d = factor((int)(e2[j] & 0xFFFFu) - (int)top) |
                                           factor((int)(e2[j] >> 16) - (int)top) << 16;
                        if (j == 0) d0 = d;
                        else d1 = d;
                    }
                    special = __any_sync(kFull, special);
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        const float f = __shfl_sync(kFull, back[k & 1], k >> 1);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int c = 0; c < 4; ++c) o[k][hh][n][c] *= f;
                    }
                } else {  // factor(e - R), both halves at once
                    d0 = d0 * 1024u + (uint32_t)(15 - kUp) * 0x04000400u;
                    d1 = d1 * 1024u + (uint32_t)(15 - kUp) * 0x04000400u;
                }
                if (special) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t half = 0xFFFFu << (16 * e);
                        if (((e2[0] >> (16 * e)) & 0xFFFFu) == 255u) d0 = (d0 & ~half) | (0x7E007E00u & half);
                        if (((e2[1] >> (16 * e)) & 0xFFFFu) == 255u) d1 = (d1 & ~half) | (0x7E007E00u & half);
                    }
                }
                *(uint2 *)(vf + vpair * NB + 2 * vhalf) = make_uint2(d0, d1);
            }
            __syncwarp();

            // 16 tokens at a time, not unrolled: the body has to stay small for
            // the instruction cache (12 warps run it out of step)
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                const uint32_t at = base + lane_off + 2 * u * (NB * 128);
                // --- S^T = K Q^T
                float sc[NT][4];
                float f0[NB], f1[NB];  // scales of tokens g and g + 8
                if constexpr (NB == 4) {
                    *(float4 *)f0 = *(const float4 *)(kf + 4 * (16 * u + g));
                    *(float4 *)f1 = *(const float4 *)(kf + 4 * (16 * u + g + 8));
                } else {
                    *(float2 *)f0 = *(const float2 *)(kf + 2 * (16 * u + g));
                    *(float2 *)f1 = *(const float2 *)(kf + 2 * (16 * u + g + 8));
                }
#pragma unroll
                for (int kk = 0; kk < NB / 2; ++kk) {
                    uint32_t r[4];  // (octet 0, 1) of block 2kk, then of block 2kk + 1
                    ldsm4(r, at + 2 * kk * 128);
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        const int k = 2 * kk + k2;
                        uint32_t ha[4], hb[4];
                        codes_f16(r[2 * k2], ha);
                        codes_f16(r[2 * k2 + 1], hb);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float c[4];
                            mma_f16_0(c, ha[0], hb[0], ha[1], hb[1], qf[n][k][0], qf[n][k][1]);
                            mma_f16(c, ha[2], hb[2], ha[3], hb[3], qf[n][k][2], qf[n][k][3]);
                            sc[n][0] = k == 0 ? c[0] * f0[k] : fmaf(c[0], f0[k], sc[n][0]);
                            sc[n][1] = k == 0 ? c[1] * f0[k] : fmaf(c[1], f0[k], sc[n][1]);
                            sc[n][2] = k == 0 ? c[2] * f1[k] : fmaf(c[2], f1[k], sc[n][2]);
                            sc[n][3] = k == 0 ? c[3] * f1[k] : fmaf(c[3], f1[k], sc[n][3]);
                        }
                    }
                }
                // --- log2 domain, masks
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) sc[n][c] *= mul[n][c & 1];
                if (edge) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int i = 16 * u + 8 * (c >> 1) + g, tk = tok0 + i;
                            if (tk >= hi[n][c & 1] || tk < lo[n][c & 1] || !((live >> i) & 1u))
                                sc[n][c] = -INFINITY;
                        }
                }
                // --- running maximum
                bool grew = false;
                float mx[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v = fmaxf(sc[n][c], sc[n][c + 2]);
                        v = fmaxf(v, __shfl_xor_sync(kFull, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(kFull, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(kFull, v, 16));
                        mx[n][c] = fmaxf(m[n][c], v - (float)kUp);
                        grew |= mx[n][c] > m[n][c];
                    }
                if (__any_sync(kFull, grew)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float f = mx[n][c] == -INFINITY ? 1.f : ex2(m[n][c] - mx[n][c]);
                            m[n][c] = mx[n][c];
                            ms[n][c] = mx[n][c] == -INFINITY ? 0.f : mx[n][c];
                            l[n][c] *= f;
                            lc[n][c] *= f;
#pragma unroll
                            for (int k = 0; k < NB; ++k)
#pragma unroll
                                for (int hh = 0; hh < 2; ++hh) {
                                    o[k][hh][n][c] *= f;
                                    o[k][hh][n][c + 2] *= f;
                                }
                        }
                }
                // --- weights of tokens (2t, 2t + 1) of octets 0 and 1, column g
                uint32_t pt[NT][2], pv[NT][2][NB];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float p[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) p[c] = ex2(sc[n][c] - ms[n][c & 1]);
                    add_to(l[n][0], lc[n][0], p[0] + p[2]);
                    add_to(l[n][1], lc[n][1], p[1] + p[3]);
                    pt[n][0] = transpose8(pack_f16(p[0], p[1]));
                    pt[n][1] = transpose8(pack_f16(p[2], p[3]));
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t f[NB];  // factors of the same tokens
                    const uint32_t *src = vf + (8 * u + 4 * q + t) * NB;
                    if constexpr (NB == 4) *(uint4 *)f = *(const uint4 *)src;
                    else *(uint2 *)f = *(const uint2 *)src;
#pragma unroll
                    for (int k = 0; k < NB; ++k)
#pragma unroll
                        for (int n = 0; n < NT; ++n) pv[n][q][k] = mul_f16x2(pt[n][q], f[k]);
                    if (special) {  // a NaN value is one for every column that sees it, however small its
                                    // weight, and none for the others
                        const int i = 16 * u + 8 * q + 2 * t;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {  // bounds of column g
                            const int h0 = __shfl_sync(kFull, hi[n][0], g >> 1), h1 = __shfl_sync(kFull, hi[n][1], g >> 1);
                            const int l0 = __shfl_sync(kFull, lo[n][0], g >> 1), l1 = __shfl_sync(kFull, lo[n][1], g >> 1);
                            const int to = g & 1 ? h1 : h0, from = g & 1 ? l1 : l0;
                            uint32_t keep = 0u;
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (tok0 + i + e < to && tok0 + i + e >= from && ((live >> (i + e)) & 1u))
                                    keep |= 0xFFFFu << (16 * e);
#pragma unroll
                            for (int k = 0; k < NB; ++k) pv[n][q][k] &= keep;
                        }
                    }
                }
                // --- O^T += V^T P^T
#pragma unroll
                for (int kk = 0; kk < NB / 2; ++kk) {
                    uint32_t r[4];  // (octet 0, 1) of block 2kk, then of block 2kk + 1
                    ldsm4_t(r, at + C::kCode + 2 * kk * 128);
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
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[st]);
        }

        // --- the 4 warps' results: o, m, l of each column
        float back[NB];  // 2^(R - 127) / 2^15
#pragma unroll
        for (int k = 0; k < NB; ++k)
            back[k] = exp2f((float)(max_exp(__shfl_sync(kFull, r15[k & 1], k >> 1)) - 142));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = l[n][c] - lc[n][c];
                v += __shfl_xor_sync(kFull, v, 4);
                v += __shfl_xor_sync(kFull, v, 8);
                v += __shfl_xor_sync(kFull, v, 16);
                const int col = 8 * n + 2 * t + c;
                if (g == 0) {
                    s_m[wid * NC + col] = m[n][c];
                    s_l[wid * NC + col] = v * (1.f / (1 << kUp));
                }
                float *dst = s_o + (wid * NC + col) * C::kOStride + 4 * g;
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    const float f = back[k];  // 2^(R - 127) / 2^15
                    *(float4 *)(dst + 32 * k) =
                        make_float4(o[k][0][n][c] * f, o[k][0][n][c + 2] * f, o[k][1][n][c] * f,
                                    o[k][1][n][c + 2] * f);
                }
            }
        consumers_sync();
        const bool done = it.parts == 1;
        float *rec = recs + ((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * C::kRec;
        if (tid == 0 && it.starts && it.parts > 1) {
            cut->q0 = s.q0;
            cut->c0 = c0;
            cut->ncol = s.ncol;
            cut->head = h;
            cut->parts = it.parts;
        }
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
                store_out(a, s.q0 + (c0 + col) / a.group, h * a.group + (c0 + col) % a.group, D, d, o0, o1,
                          mt, lt, kUp);
            }
        }
        consumers_sync();  // the merge buffer is read before the next item's results come
    }
}

// Joins the partial results of the item that CTA blockIdx.x of the split
// kernel began and did not finish, always in the same order: each of 8 warps
// takes every eighth part, the loads of four in flight, and the warps' sums are joined in warp order.
constexpr int kJoinWarps = 8, kJoinCols = 2;
template <int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) moe_attn_join_kernel(MoeAttnArgs a) {
    using C = Cfg<D, NT>;
    constexpr int NC = kJoinCols, V = NC * D / 128;  // columns of a block; float4s of a lane
    __shared__ float4 s_o[kJoinWarps][V][32];
    __shared__ float s_m[kJoinWarps][NC], s_l[kJoinWarps][NC];
    grid_dep_wait();
    grid_dep_launch();
    const Cut cut = ((const Cut *)a.part)[blockIdx.x];
    const int col0 = NC * blockIdx.y;
    if (cut.parts == 0 || cut.c0 + col0 >= cut.ncol) return;
    const float *recs = a.part + (size_t)gridDim.x * C::kHead;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    auto rec = [&](int p) {
        return recs + ((int64_t)(blockIdx.x + p) * 2 + (p == 0 ? 1 : 0)) * C::kRec;
    };
    // float4 i of a lane belongs to column (32 i + lane) / (D / 4)
    float mt[V], lt[V];
    float4 o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) mt[i] = -INFINITY, lt[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = wid; p < cut.parts; p += kJoinWarps) {
        const float *r = rec(p);
        float4 v[V];
        float mp[V], lp[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = col0 + (32 * i + lane) / (D / 4);
            v[i] = ((const float4 *)(r + col0 * D))[32 * i + lane];
            mp[i] = r[C::NC * D + col];
            lp[i] = r[C::NC * D + C::NC + col];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float mn = fmaxf(mt[i], mp[i]), sf = mn == -INFINITY ? 0.f : mn;
            const float f = ex2(mt[i] - sf), w = ex2(mp[i] - sf);
            mt[i] = mn;
            lt[i] = fmaf(lt[i], f, w * lp[i]);
            o[i].x = fmaf(o[i].x, f, w * v[i].x);
            o[i].y = fmaf(o[i].y, f, w * v[i].y);
            o[i].z = fmaf(o[i].z, f, w * v[i].z);
            o[i].w = fmaf(o[i].w, f, w * v[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s_o[wid][i][lane] = o[i];
        const int x = 32 * i + lane;
        if (x % (D / 4) == 0) {
            s_m[wid][x / (D / 4)] = mt[i];
            s_l[wid][x / (D / 4)] = lt[i];
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < NC * D / 2; x += 32 * kJoinWarps) {
        const int col = x / (D / 2), d = x % (D / 2) * 2, c = cut.c0 + col0 + col;
        if (c >= cut.ncol) continue;
        float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_m[w][col]);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float f = s_m[w][col] == -INFINITY ? 0.f : ex2(s_m[w][col] - m);
            const float2 v = ((const float2 *)&s_o[w][0][0])[x];
            l = fmaf(f, s_l[w][col], l);
            o0 = fmaf(f, v.x, o0);
            o1 = fmaf(f, v.y, o1);
        }
        store_out(a, cut.q0 + c / a.group, cut.head * a.group + c % a.group, D, d, o0, o1, m, l, kUp);
    }
}

// Two column tiles of 8 where a sequence may have more than 8 columns.
bool wide(int group, int max_q) { return (int64_t)group * max_q > 8; }

// A CTA takes whole items where each has at most a tile per warp, and nothing is
// left to join: 48 sequences of 128 keys 9.0 us, on the line 10.5.
bool whole_items(int max_kv) { return max_kv <= kWarps * kTile; }

template <int D, int NT>
cudaError_t launch(const MoeAttnArgs &a, int nsm, cudaStream_t st) {
    using C = Cfg<D, NT>;
    const bool whole = whole_items(a.b.max_kv);
    // no more CTAs than the bounds allow items, or parts of the least size
    const int64_t items = (int64_t)a.n_kv * ((int64_t)a.b.n_tokens * a.group / C::NC + a.b.n_seqs);
    const int64_t parts = whole ? 1 : (a.b.max_kv / kTile + 2 + kMinTiles - 1) / kMinTiles;
    const int ctas = (int)std::min<int64_t>(items * parts, (int64_t)nsm * C::kCtasPerSm);
    const cudaError_t err = launch_pdl_ready(moe_attn_split_kernel<D, NT>, dim3(ctas), dim3(kThreads), C::kSmem, st, a, whole);
    if (err != cudaSuccess || whole) return err;
    return launch_pdl_ready(moe_attn_join_kernel<D, NT>, dim3(ctas, C::NC / kJoinCols), dim3(32 * kJoinWarps), 0, st, a);
}

template <int D, int NT>
cudaError_t setup() {
    const cudaError_t err = set_kernel((const void *)moe_attn_split_kernel<D, NT>, Cfg<D, NT>::kSmem);
    return err != cudaSuccess ? err : set_kernel((const void *)moe_attn_join_kernel<D, NT>);
}

}  // namespace

cudaError_t moe_attn_setup() {
    cudaError_t err = setup<64, 1>();
    if (err == cudaSuccess) err = setup<64, 2>();
    if (err == cudaSuccess) err = setup<128, 1>();
    if (err == cudaSuccess) err = setup<128, 2>();
    return err != cudaSuccess ? err : moe_attn_prefill_setup();
}

size_t moe_attn_ws_bytes(int head_dim, int group, int max_q, int max_kv, int nsm) {
    auto split = [&](int nt, int per_sm) {
        return (size_t)nsm * per_sm * (2 * (8 * nt * (head_dim + 2)) + 8) * sizeof(float);
    };
    // (never less for larger bounds: a batch within them may go either way)
    const size_t one = whole_items(max_kv) ? 0 : split(1, 3);
    const size_t two = whole_items(max_kv) || !wide(group, max_q) ? 0 : split(2, 2);
    return std::max({one, two, moe_attn_prefill_ws_bytes(head_dim, group, max_q, max_kv, nsm)});
}

cudaError_t moe_launch_attn(int head_dim, const MoeAttnArgs &a, int nsm, cudaStream_t st) {
    if (moe_attn_prefill_fits(a.b.n_seqs, a.n_kv, a.group, a.b.max_q, a.b.max_kv))
        return moe_launch_attn_prefill(head_dim, a, nsm, st);
    const bool w = wide(a.group, a.b.max_q);
    if (head_dim == 64) return w ? launch<64, 2>(a, nsm, st) : launch<64, 1>(a, nsm, st);
    return w ? launch<128, 2>(a, nsm, st) : launch<128, 1>(a, nsm, st);
}
