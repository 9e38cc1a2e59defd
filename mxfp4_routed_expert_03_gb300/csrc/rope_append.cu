// Norm and rotation of queries and keys with the keys and values going straight
// into the MXFP4 cache, in one launch.
//
// Per head row the mathematics of qk_rope.cu (rope.cuh), keys rounded once to
// bf16, then per 32 elements that of kv_cache.cu (kv_block.cuh): the same bits as
// the two calls, without the keys' way through memory. Bound: 2 bytes read per
// element, 2 written for queries and 17/32 for keys and values; 8191 tokens of 56
// query and 8 + 8 key and value heads of 128 49 us (5.7 TB/s of the 277 MB; 56.6
// with ordinary loads, see cp_async_16; the two calls take 61.7).
//
// A warp has one of three kinds of task: TOK tokens' keys of one head (normed and
// rotated in two passes of the row layout, exchanged through 2 KB of shared memory
// into the cache's layout of one block per lane, so that its code store is 512
// consecutive bytes when the slots are consecutive), the same tokens' values of one
// head, or query rows of one token as in qk_rope.cu. Keys and values come first:
// their chain is the longest.
#include "kv_block.cuh"
#include "rope.cuh"

namespace {

constexpr int kWarps = 4;

// A warp's query rows: P passes of 32 / (D / 16) of them, all on their way to shared memory at once, each
// lane copying the chunks that it reads itself.
template <int D, int P>
__global__ void __launch_bounds__(32 * kWarps)
    moe_rope_append_kernel(MoeRopeArgs a, MoeKvArgs c, int groups, uint32_t kv_tasks) {
    constexpr int TPH = D / 16;            // threads per head row
    constexpr int HP = 32 / TPH;           // head rows per warp and pass
    constexpr int NB = D / 32;             // blocks of a head row
    constexpr int TOK = 32 / NB;           // tokens of a key or value task
    static_assert(TOK == 2 * HP && TOK * D / 8 == 128, "two passes per key task");
    static_assert(P * 64 <= 256, "room for the rows");
    __shared__ uint4 space[kWarps][256];
    const int lane = threadIdx.x & 31;
    uint4 *mine = space[threadIdx.x >> 5] + lane;
    uint32_t task = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const rope::Lane l(lane % TPH, a.rope_dim);
    grid_dep_wait();
    grid_dep_launch();
    if (task < 2 * kv_tasks) {
        const bool is_v = task >= kv_tasks;
        if (is_v) task -= kv_tasks;
        const int first = (int)(task / c.n_kv) * TOK, head = (int)(task % c.n_kv);
        // the block that this lane writes: block b of token `tok`
        const int b = lane / 8 % NB, to = lane / (8 * NB) * 8 + lane % 8, tok = first + to;
        int slot = -1, at = 0;
        uint32_t w[16];
        if (is_v) {
            if (tok >= c.n) return;
            const uint16_t *src = c.v + (int64_t)tok * c.v_stride + head * D + 32 * b;
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async_16(mine + 32 * i, src + 8 * i);
            cp_async_commit();
            slot = c.slots[tok];
            if (a.rope_dim > 0) at = a.positions[tok];
            cp_async_wait<0>();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 x = mine[32 * i];
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
        } else {
            int pos[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int t = first + p * HP + lane / TPH;
                pos[p] = 0;
                if (t >= c.n) {
                    mine[64 * p] = mine[64 * p + 32] = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    const uint16_t *src = a.k + (int64_t)t * a.k_stride + head * D;
                    cp_async_16(mine + 64 * p, src + 8 * l.c0);
                    cp_async_16(mine + 64 * p + 32, src + 8 * l.c1);
                    if (a.rope_dim > 0) pos[p] = a.positions[t];
                }
            }
            cp_async_commit();
            if (tok < c.n) {
                slot = c.slots[tok];
                if (a.rope_dim > 0) at = a.positions[tok];
            }
            cp_async_wait<0>();
            uint4 *stage = space[threadIdx.x >> 5] + 128;  // [TOK rows][D / 8 chunks]
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int r = p * HP + lane / TPH;
                float x[8], y[8], cs[8], sn[8];
                rope::unpack8(mine[64 * p], x);
                rope::unpack8(mine[64 * p + 32], y);
                const float ss = rope::row_squares<D>(x, y);
                // (rows of a bad position are not turned, nor written below)
                const bool ok = pos[p] >= 0 && pos[p] < a.n_pos;
                rope::Lane turned = l;
                turned.turn = l.turn && ok;
                if (turned.turn) rope::load_angles(a, l, pos[p], cs, sn);
                rope::norm_turn<D>(a, turned, a.k_weight, ss, cs, sn, x, y);
                // 16-byte chunks permuted by the row, so that neither side's accesses collide
                stage[r * (D / 8) + (l.c0 ^ (r & 7))] = rope::pack8(x);
                stage[r * (D / 8) + (l.c1 ^ (r & 7))] = rope::pack8(y);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 x = stage[to * (D / 8) + ((4 * b + i) ^ (to & 7))];
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
            if (tok >= c.n) return;
        }
        if (a.rope_dim > 0 && (at < 0 || at >= a.n_pos)) {
            moe_flag(a.status, MOE_ERR_BAD_INDEX);
            return;
        }
        if (kv::slot_ok(c, slot)) kv::write_block<NB>(c, is_v, slot, head, b, w);
        return;
    }
    task -= 2 * kv_tasks;
    const uint32_t token = task / groups, group = task - token * groups;
    if (token >= (uint32_t)c.n) return;
    const int64_t t = token;
    const int row0 = group * P * HP + lane / TPH;
    const int pos = a.rope_dim > 0 ? a.positions[t] : 0;  // (in flight beside the rows)
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int r = row0 + p * HP;
        if (r < a.n_q) {
            const uint16_t *src = a.q + t * a.q_stride + (int64_t)r * D;
            cp_async_16(mine + 64 * p, src + 8 * l.c0);
            cp_async_16(mine + 64 * p + 32, src + 8 * l.c1);
        }
    }
    cp_async_commit();
    if (a.rope_dim > 0 && (pos < 0 || pos >= a.n_pos)) {
        if (lane == 0 && group == 0) moe_flag(a.status, MOE_ERR_BAD_INDEX);
        cp_async_wait<0>();
        return;
    }
    float cs[8], sn[8];
    if (l.turn) rope::load_angles(a, l, pos, cs, sn);
    cp_async_wait<0>();
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int r = row0 + p * HP;
        float x[8], y[8];
        // (rows that are not there hold what was in shared memory, and end here)
        rope::unpack8(mine[64 * p], x);
        rope::unpack8(mine[64 * p + 32], y);
        const float ss = rope::row_squares<D>(x, y);
        if (r >= a.n_q) continue;
        rope::norm_turn<D>(a, l, a.q_weight, ss, cs, sn, x, y);
        uint16_t *dst = a.q_out + t * a.q_out_stride + (int64_t)r * D;
        *(uint4 *)(dst + 8 * l.c0) = rope::pack8(x);
        *(uint4 *)(dst + 8 * l.c1) = rope::pack8(y);
    }
}

template <int D, int P>
cudaError_t launch(const MoeRopeArgs &a, const MoeKvArgs &c, cudaStream_t st) {
    constexpr int TOK = 1024 / D;
    const int per_warp = P * (32 / (D / 16)), groups = (a.n_q + per_warp - 1) / per_warp;
    const uint32_t kv_tasks = (uint32_t)((c.n + TOK - 1) / TOK) * c.n_kv;
    const int64_t tasks = 2 * (int64_t)kv_tasks + (int64_t)c.n * groups;
    return launch_pdl_ready(moe_rope_append_kernel<D, P>, dim3((unsigned)((tasks + kWarps - 1) / kWarps)),
                            dim3(32 * kWarps), 0, st, a, c, groups > 0 ? groups : 1, kv_tasks);
}

// Query rows of a warp: one pass for few tokens (as qk_rope.cu), else four (8191 tokens of 56 + 16 heads of 128: 2
// passes 50.9 us, 4 48.9, 8 51.4; 7000 of 64 + 16 53.8, 54.5, 59.5; 400 of 56 + 16 5.2, 4.9, 6.1).
template <int D>
cudaError_t launch(const MoeRopeArgs &a, const MoeKvArgs &c, int nsm, cudaStream_t st) {
    return (int64_t)c.n * a.n_q < (int64_t)nsm * 64 ? launch<D, 1>(a, c, st) : launch<D, 4>(a, c, st);
}

}  // namespace

cudaError_t moe_rope_append_setup() {
    const void *kernels[] = {
        (const void *)moe_rope_append_kernel<64, 1>, (const void *)moe_rope_append_kernel<64, 4>,
        (const void *)moe_rope_append_kernel<128, 1>, (const void *)moe_rope_append_kernel<128, 4>};
    for (const void *k : kernels) {
        const cudaError_t err = set_kernel(k);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

cudaError_t moe_launch_rope_append(int head_dim, const MoeRopeArgs &a, const MoeKvArgs &c, int nsm,
                                   cudaStream_t st) {
    return head_dim == 64 ? launch<64>(a, c, nsm, st) : launch<128>(a, c, nsm, st);
}
