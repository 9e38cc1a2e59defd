// C ABI of the attention operators: argument validation and launches. See
// include/moe.h for the contract.
#include <stdlib.h>

#include "api_util.h"
#include "common.cuh"
#include "kernels.h"

struct moe_attn {
    moe_attn_desc desc;
    moe_kv_cache cache;
    int page_shift;  // log2(page_size)
    int device;
    int num_sms;
    int *status;     // device word: first error code recorded by a kernel
    int inject;      // enum moe_inject (test hook; MOE_INJECT_NONE by default)
    long long timeout;
};

static int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// MOE_OK, or why the shape is refused.
static int check_desc(const moe_attn_desc *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->n_heads <= 0 || d->n_kv_heads <= 0 || d->head_dim <= 0 || d->page_size <= 0 ||
        d->n_pages <= 0 || d->n_heads % d->n_kv_heads)
        return MOE_ERR_INVALID_ARG;
    if (d->n_heads > 1024 || (d->head_dim != 64 && d->head_dim != 128) ||
        page_shift_of(d->page_size) < 0 || (int64_t)d->n_pages * d->page_size > INT32_MAX)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

MOE_API int64_t moe_kv_code_bytes(const moe_attn_desc *d) {
    if (check_desc(d) != MOE_OK) return -1;
    return (int64_t)d->n_pages * d->n_kv_heads * d->page_size * (d->head_dim / 2);
}

MOE_API int64_t moe_kv_scale_bytes(const moe_attn_desc *d) {
    if (check_desc(d) != MOE_OK) return -1;
    return (int64_t)d->n_pages * d->n_kv_heads * d->page_size * (d->head_dim / 32);
}

MOE_API int moe_attn_create(const moe_attn_desc *d, const moe_kv_cache *c, moe_attn **out) {
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = NULL;
    if (!d || !c) return MOE_ERR_INVALID_ARG;
    const int rc = check_desc(d);
    if (rc != MOE_OK) return rc;
    const void *arrays[] = {c->k_q, c->k_s, c->v_q, c->v_s};
    for (const void *p : arrays)
        if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;  // bulk copies
    int dev = 0, major = 0, minor = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;
    if (moe_qk_norm_rope_setup() != cudaSuccess || moe_kv_setup() != cudaSuccess ||
        moe_rope_append_setup() != cudaSuccess || moe_attn_setup() != cudaSuccess)
        return MOE_ERR_CUDA;
    moe_attn *a = (moe_attn *)calloc(1, sizeof(moe_attn));
    if (!a) return MOE_ERR_INVALID_ARG;
    a->desc = *d;
    a->cache = *c;
    a->page_shift = page_shift_of(d->page_size);
    a->device = dev;
    a->num_sms = nsm;
    a->inject = MOE_INJECT_NONE;
    a->timeout = kTimeoutCycles;
    if (cudaMalloc(&a->status, sizeof(int)) != cudaSuccess) {
        free(a);
        return MOE_ERR_CUDA;
    }
    if (cudaMemset(a->status, 0, sizeof(int)) != cudaSuccess) {
        cudaFree(a->status);
        free(a);
        return MOE_ERR_CUDA;
    }
    *out = a;
    return MOE_OK;
}

MOE_API void moe_attn_destroy(moe_attn *a) {
    if (!a) return;
    cudaFree(a->status);
    free(a);
}

// A strided bf16 array of token rows of `width` elements: 16-byte vectors.
static bool rows_ok(const void *p, int64_t stride, int64_t width) {
    return p && aligned16(p) && stride % 8 == 0 && stride >= width;
}

// Whether norm and rotation parameters make sense, tokens or not.
static bool rope_desc_ok(const moe_attn_desc &d, const moe_rope_desc *r) {
    return r->rope_dim >= 0 && r->rope_dim <= d.head_dim && r->rope_dim % 16 == 0 && r->n_pos >= 0 &&
           (r->interleaved == 0 || r->interleaved == 1) && finite_f32(r->eps) && r->eps >= 0.f &&
           aligned16(r->q_weight) && aligned16(r->k_weight);
}

// Whether a rotation has its table and positions.
static bool rope_arrays_ok(const moe_rope_desc *r, const int32_t *positions) {
    return r->rope_dim == 0 ||
           (r->cos_sin && aligned16(r->cos_sin) && positions && !((uintptr_t)positions & 3u));
}

static MoeRopeArgs rope_args(const moe_attn *a, const moe_rope_desc *r, const int32_t *positions,
                             const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                             uint16_t *q_out, int64_t q_out_stride) {
    MoeRopeArgs g = {};
    g.n_q = q ? a->desc.n_heads : 0;
    g.n_k = k ? a->desc.n_kv_heads : 0;
    g.rope_dim = r->rope_dim;
    g.interleaved = r->interleaved;
    g.n_pos = r->n_pos;
    g.eps = r->eps;
    g.cos_sin = r->cos_sin;
    g.q_weight = r->q_weight;
    g.k_weight = r->k_weight;
    g.positions = positions;
    g.q = q;
    g.k = k;
    g.q_out = q_out;
    g.q_stride = q_stride;
    g.k_stride = k_stride;
    g.q_out_stride = q_out_stride;
    g.status = a->status;
    return g;
}

MOE_API int moe_qk_norm_rope(moe_attn *a, int32_t T, const moe_rope_desc *r,
                             const int32_t *positions, const uint16_t *q, int64_t q_stride,
                             const uint16_t *k, int64_t k_stride, uint16_t *q_out,
                             int64_t q_out_stride, uint16_t *k_out, int64_t k_out_stride,
                             void *stream) {
    NvtxRange nvtx_range("moe_qk_norm_rope");
    if (!a || T < 0 || !r) return MOE_ERR_INVALID_ARG;
    const moe_attn_desc &d = a->desc;
    if (!rope_desc_ok(d, r)) return MOE_ERR_INVALID_ARG;
    if ((!q) != (!q_out) || (!k) != (!k_out)) return MOE_ERR_INVALID_ARG;
    if (T == 0 || (!q && !k)) return MOE_OK;
    if (!rope_arrays_ok(r, positions)) return MOE_ERR_INVALID_ARG;
    const int64_t qw = (int64_t)d.n_heads * d.head_dim, kw = (int64_t)d.n_kv_heads * d.head_dim;
    if (q && (!rows_ok(q, q_stride, qw) || !rows_ok(q_out, q_out_stride, qw)))
        return MOE_ERR_INVALID_ARG;
    if (k && (!rows_ok(k, k_stride, kw) || !rows_ok(k_out, k_out_stride, kw)))
        return MOE_ERR_INVALID_ARG;
    if ((int64_t)T * (d.n_heads + d.n_kv_heads) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    MoeRopeArgs g = rope_args(a, r, positions, q, q_stride, k, k_stride, q_out, q_out_stride);
    g.k_out = k_out;
    g.k_out_stride = k_out_stride;
    return moe_launch_qk_norm_rope(T, d.head_dim, g, a->num_sms, (cudaStream_t)stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

static MoeKvArgs kv_args(const moe_attn *a, int n, const int32_t *slots) {
    MoeKvArgs g = {};
    g.n = n;
    g.n_kv = a->desc.n_kv_heads;
    g.n_slots = a->desc.n_pages * a->desc.page_size;
    g.page_shift = a->page_shift;
    g.slots = slots;
    g.c = a->cache;
    g.status = a->status;
    return g;
}

MOE_API int moe_kv_append(moe_attn *a, int32_t T, const uint16_t *k, int64_t k_stride,
                          const uint16_t *v, int64_t v_stride, const int32_t *slots, void *stream) {
    NvtxRange nvtx_range("moe_kv_append");
    if (!a || T < 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const int64_t w = (int64_t)a->desc.n_kv_heads * a->desc.head_dim;
    if (!rows_ok(k, k_stride, w) || !rows_ok(v, v_stride, w) || !slots || ((uintptr_t)slots & 3u))
        return MOE_ERR_INVALID_ARG;
    if ((int64_t)T * a->desc.n_kv_heads > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    MoeKvArgs g = kv_args(a, T, slots);
    g.k = k;
    g.v = v;
    g.k_stride = k_stride;
    g.v_stride = v_stride;
    return moe_launch_kv_append(a->desc.head_dim, g, (cudaStream_t)stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

MOE_API int moe_rope_append(moe_attn *a, int32_t T, const moe_rope_desc *r,
                            const int32_t *positions, const uint16_t *q, int64_t q_stride,
                            const uint16_t *k, int64_t k_stride, const uint16_t *v,
                            int64_t v_stride, const int32_t *slots, uint16_t *q_out,
                            int64_t q_out_stride, void *stream) {
    NvtxRange nvtx_range("moe_rope_append");
    if (!a || T < 0 || !r || !rope_desc_ok(a->desc, r) || (!q) != (!q_out)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const moe_attn_desc &d = a->desc;
    const int64_t qw = (int64_t)d.n_heads * d.head_dim, kw = (int64_t)d.n_kv_heads * d.head_dim;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != a->device) return MOE_ERR_INVALID_ARG;
    if (!rope_arrays_ok(r, positions) || !rows_ok(k, k_stride, kw) || !rows_ok(v, v_stride, kw) || !slots ||
        ((uintptr_t)slots & 3u) || (q && (!rows_ok(q, q_stride, qw) || !rows_ok(q_out, q_out_stride, qw))))
        return MOE_ERR_INVALID_ARG;
    if ((int64_t)T * (d.n_heads + 2 * d.n_kv_heads) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    MoeKvArgs c = kv_args(a, T, slots);
    c.v = v;
    c.v_stride = v_stride;
    const MoeRopeArgs g = rope_args(a, r, positions, q, q_stride, k, k_stride, q_out, q_out_stride);
    return moe_launch_rope_append(d.head_dim, g, c, a->num_sms, (cudaStream_t)stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

MOE_API int moe_kv_read(moe_attn *a, int32_t n, const int32_t *slots, uint16_t *k, int64_t k_stride,
                        uint16_t *v, int64_t v_stride, void *stream) {
    NvtxRange nvtx_range("moe_kv_read");
    if (!a || n < 0) return MOE_ERR_INVALID_ARG;
    if (n == 0 || (!k && !v)) return MOE_OK;
    const int64_t w = (int64_t)a->desc.n_kv_heads * a->desc.head_dim;
    if ((k && !rows_ok(k, k_stride, w)) || (v && !rows_ok(v, v_stride, w)) || !slots ||
        ((uintptr_t)slots & 3u))
        return MOE_ERR_INVALID_ARG;
    if ((int64_t)n * a->desc.n_kv_heads > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    MoeKvArgs g = kv_args(a, n, slots);
    g.k_out = k;
    g.v_out = v;
    g.k_stride = k_stride;
    g.v_stride = v_stride;
    return moe_launch_kv_read(a->desc.head_dim, g, (cudaStream_t)stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

static bool bounds_ok(int n_seqs, int n_tokens, int max_q, int max_kv) {
    return n_seqs >= 0 && n_tokens >= 0 && max_q >= 0 && max_kv >= 0;
}

MOE_API size_t moe_attn_workspace_bytes(const moe_attn *a, int32_t n_seqs, int32_t n_tokens,
                                        int32_t max_q, int32_t max_kv) {
    if (!a || !bounds_ok(n_seqs, n_tokens, max_q, max_kv) || n_seqs == 0 || n_tokens == 0) return 0;
    return align_up(moe_attn_ws_bytes(a->desc.head_dim, a->desc.n_heads / a->desc.n_kv_heads, max_q,
                                      max_kv, a->num_sms),
                    256);
}

MOE_API int moe_attn_forward(moe_attn *a, const moe_attn_batch *b, const uint16_t *q,
                             int64_t q_stride, uint16_t *out, int64_t out_stride, float *lse,
                             void *ws, size_t ws_bytes, void *stream) {
    NvtxRange nvtx_range("moe_attn_forward");
    if (!a || !b || !bounds_ok(b->n_seqs, b->n_tokens, b->max_q, b->max_kv))
        return MOE_ERR_INVALID_ARG;
    if (b->window < 0 || !finite_f32(b->scale)) return MOE_ERR_INVALID_ARG;
    if (b->n_seqs == 0 || b->n_tokens == 0) return MOE_OK;
    const moe_attn_desc &d = a->desc;
    const int64_t w = (int64_t)d.n_heads * d.head_dim;
    if (!rows_ok(q, q_stride, w) || !rows_ok(out, out_stride, w) || ((uintptr_t)lse & 3u))
        return MOE_ERR_INVALID_ARG;
    if (!b->cu_q && b->n_tokens != b->n_seqs) return MOE_ERR_INVALID_ARG;
    if (!b->kv_len || b->max_q < 1) return MOE_ERR_INVALID_ARG;
    if (((uintptr_t)b->cu_q | (uintptr_t)b->kv_len | (uintptr_t)b->page_table) & 3u)
        return MOE_ERR_INVALID_ARG;
    if (b->max_kv > 0 &&
        (!b->page_table || ((int64_t)b->max_kv + d.page_size - 1) / d.page_size > b->table_stride))
        return MOE_ERR_INVALID_ARG;
    // 32-bit token positions with room for a tile, and rows x heads
    if (b->max_kv > INT32_MAX - 65536 || b->window > INT32_MAX / 2 ||
        (int64_t)b->n_tokens * d.n_heads > INT32_MAX / 2)
        return MOE_ERR_UNSUPPORTED;
    const size_t need = moe_attn_workspace_bytes(a, b->n_seqs, b->n_tokens, b->max_q, b->max_kv);
    if (ws_bytes < need || (need && (!ws || ((uintptr_t)ws & 255u)))) return MOE_ERR_WORKSPACE;
    MoeAttnArgs g = {};
    g.n_kv = d.n_kv_heads;
    g.group = d.n_heads / d.n_kv_heads;
    g.page_shift = a->page_shift;
    g.n_pages = d.n_pages;
    g.c = a->cache;
    g.b = *b;
    g.q = q;
    g.q_stride = q_stride;
    g.out = out;
    g.out_stride = out_stride;
    g.lse = lse;
    g.part = (float *)ws;
    g.status = a->status;
    g.timeout_cycles = a->timeout;
    g.inject = a->inject;
    return moe_launch_attn(d.head_dim, g, a->num_sms, (cudaStream_t)stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

MOE_API int moe_attn_set_fault_injection(moe_attn *a, int32_t mode, int64_t timeout_cycles) {
    if (!a || (mode != MOE_INJECT_NONE && mode != MOE_INJECT_ATTN_STALL)) return MOE_ERR_INVALID_ARG;
    if (timeout_cycles > 0 && timeout_cycles < 100000) return MOE_ERR_INVALID_ARG;
    a->inject = mode;
    a->timeout = timeout_cycles > 0 ? (long long)timeout_cycles : kTimeoutCycles;
    return MOE_OK;
}

MOE_API int moe_attn_status(moe_attn *a, void *stream) {
    if (!a) return MOE_ERR_INVALID_ARG;
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return MOE_ERR_CUDA;
    int v = 0;
    if (cudaMemcpy(&v, a->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (v != 0 && cudaMemset(a->status, 0, sizeof(int)) != cudaSuccess) return MOE_ERR_CUDA;
    return v;
}
