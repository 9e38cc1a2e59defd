// The MXFP4 key/value cache: written token by token, read back.
//
// Per 32 elements: scale 2^e, e = floor(log2 max|x|) - 2 clamped to E8M0's
// range, elements x / 2^e rounded to the nearest E2M1 value (ties to even,
// clamped to 6): powers of two and one rounding, so codes are exact. Bound:
// 2 bytes an element on one side, 17/32 on the other.
//
// Layout: the 16-byte blocks of 8 consecutive tokens lie together (128 bytes
// per 8 tokens and 32 dimensions), which is the 8x8 tile of 16-bit units that
// ldmatrix reads: attention gets a key fragment, or a transposed value
// fragment, of packed codes with one conflict-free load.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_block.cuh"

namespace {

constexpr int kWarps = 4;

// Writing: a lane takes one block of one token (64 bytes in, 16 out), a warp 32
// / NB tokens of a head, so that its code store is 512 consecutive bytes when the
// tokens' slots are consecutive, and no lane needs another's maximum (with 4 lanes a
// block the exchange took most of the instructions: 16384 tokens x 8 heads 22 us).
template <int D>
__global__ void __launch_bounds__(32 * kWarps) moe_kv_append_kernel(MoeKvArgs a) {
    constexpr int NB = D / 32, TOK = 32 / NB;
    const int lane = threadIdx.x & 31, b = lane / 8 % NB;
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), group = unit / (2u * a.n_kv);
    const int tok = (int)group * TOK + lane / (8 * NB) * 8 + lane % 8;
    const int sub = (int)(unit - group * (2u * a.n_kv)), head = sub >> 1;
    const bool is_v = sub & 1;
    grid_dep_wait();
    grid_dep_launch();
    if (tok >= a.n) return;
    const int slot = a.slots[tok];
    const uint4 *src = (const uint4 *)((is_v ? a.v + (int64_t)tok * a.v_stride : a.k + (int64_t)tok * a.k_stride) +
                                       head * D + 32 * b);
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 x = src[i];
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
    if (!kv::slot_ok(a, slot)) return;  // (behind the loads, which do not wait for it)
    kv::write_block<NB>(a, is_v, slot, head, b, w);
}

// Two E2M1 codes (a byte) to fp32.
__device__ __forceinline__ float2 e2m1x2_to_f32(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(h)
        : "r"(byte));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// Reading: a warp takes 8 tokens of one head, 4 lanes per token, lane t of them
// elements 8t .. 8t+7 of every block, so that rows are written in 64-byte pieces.
template <int D>
__global__ void __launch_bounds__(32 * kWarps) moe_kv_read_kernel(MoeKvArgs a) {
    constexpr int NB = D / 32;
    const int lane = threadIdx.x & 31;
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), group = unit / (2u * a.n_kv);
    const int tok = (int)group * 8 + (lane >> 2);
    const int sub = (int)(unit - group * (2u * a.n_kv)), head = sub >> 1, q = lane & 3;
    const bool is_v = sub & 1;
    grid_dep_wait();
    grid_dep_launch();
    if (tok >= a.n) return;
    const int slot = a.slots[tok];
    if (!kv::slot_ok(a, slot)) return;
    uint16_t *out = is_v ? a.v_out : a.k_out;
    if (!out) return;
    out += (int64_t)tok * (is_v ? a.v_stride : a.k_stride) + head * D + 8 * q;
    const uint8_t *sq = (is_v ? a.c.v_q : a.c.k_q) + kv::code_offset<NB>(a, slot, head) + 4 * q;
    const uint8_t *ss = is_v ? a.c.v_s : a.c.k_s;
    uint32_t code[NB], byte[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        code[b] = *(const uint32_t *)(sq + 128 * b);
        byte[b] = ss[kv::scale_offset<NB>(a, slot, head, b, is_v)];
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const float s = e8m0_to_f32(byte[b]);  // value x 2^e is exact in bf16
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = e2m1x2_to_f32((code[b] >> (8 * j)) & 0xFFu);
            const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);
            w[j] = *reinterpret_cast<const uint32_t *>(&r);
        }
        *(uint4 *)(out + 32 * b) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

int blocks(const MoeKvArgs &a, int tokens) {  // `tokens` of a warp
    const int64_t units = (int64_t)((a.n + tokens - 1) / tokens) * 2 * a.n_kv;
    return (int)((units + kWarps - 1) / kWarps);
}

}  // namespace

cudaError_t moe_kv_setup() {
    const void *kernels[] = {(const void *)moe_kv_append_kernel<64>, (const void *)moe_kv_append_kernel<128>,
                             (const void *)moe_kv_read_kernel<64>, (const void *)moe_kv_read_kernel<128>};
    for (const void *k : kernels) {
        const cudaError_t err = set_kernel(k);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

cudaError_t moe_launch_kv_append(int head_dim, const MoeKvArgs &a, cudaStream_t st) {
    return head_dim == 64
               ? launch_pdl_ready(moe_kv_append_kernel<64>, dim3(blocks(a, 16)), dim3(32 * kWarps), 0, st, a)
               : launch_pdl_ready(moe_kv_append_kernel<128>, dim3(blocks(a, 8)), dim3(32 * kWarps), 0, st, a);
}

cudaError_t moe_launch_kv_read(int head_dim, const MoeKvArgs &a, cudaStream_t st) {
    return head_dim == 64
               ? launch_pdl_ready(moe_kv_read_kernel<64>, dim3(blocks(a, 8)), dim3(32 * kWarps), 0, st, a)
               : launch_pdl_ready(moe_kv_read_kernel<128>, dim3(blocks(a, 8)), dim3(32 * kWarps), 0, st, a);
}
