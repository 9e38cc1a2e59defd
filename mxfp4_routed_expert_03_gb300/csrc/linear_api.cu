// C ABI of the norm and the dense product in 8 bits: argument validation and
// launches. See include/moe.h for the contract.
#include <stdlib.h>

#include "api_util.h"
#include "common.cuh"
#include "kernels.h"
#include "tensor_map.h"

struct moe_norm {
    moe_norm_desc desc;
    int device;
    int num_sms;
};

struct moe_linear {
    moe_linear_desc desc;
    const float *w_s;
    CUtensorMap map_w, map_w64;  // boxes of 128 and of 64 weight rows
    int device;
    int num_sms;
    int *status;  // device word: first error code recorded by a kernel
    int inject;   // enum moe_inject (test hook; MOE_INJECT_NONE by default)
    long long timeout;
};

// The current device and its number of SMs, once it is known to be an sm_103.
static int check_device(int *dev, int *nsm) {
    int major = 0, minor = 0;
    if (cudaGetDevice(dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess ||
        cudaDeviceGetAttribute(nsm, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    return major == 10 && minor == 3 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

static bool current(int device) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == device;
}

// A strided array of token rows of `width` bf16 elements: 16-byte vectors.
static bool rows_ok(const void *p, int64_t stride, int64_t width) {
    return p && aligned16(p) && stride % 8 == 0 && stride >= width;
}

// `packed`: rows of an odd multiple of 8 codes, one behind the other. (With room for a multiple of 16 the product
// would take the codes behind them, which nobody writes, for part of the row.)
static bool rows8_ok(const moe_fp8_rows *r, int64_t width, bool packed = false) {
    return r->q && aligned16(r->q) && (packed ? r->q_stride == width : r->q_stride % 16 == 0 && r->q_stride >= width) &&
           r->s && !((uintptr_t)r->s & 3u) && r->s_stride >= (width + 127) / 128;
}

MOE_API int moe_norm_create(const moe_norm_desc *d, moe_norm **out) {
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = NULL;
    if (!d || d->d_model <= 0 || d->d_model % 8 || !finite_f32(d->eps) || d->eps < 0.f ||
        !aligned16(d->weight))
        return MOE_ERR_INVALID_ARG;
    if (d->d_model > MOE_NORM_MAX_D) return MOE_ERR_UNSUPPORTED;
    int dev = 0, nsm = 0;
    const int rc = check_device(&dev, &nsm);
    if (rc != MOE_OK) return rc;
    if (moe_norm_setup() != cudaSuccess) return MOE_ERR_CUDA;
    moe_norm *n = (moe_norm *)calloc(1, sizeof(moe_norm));
    if (!n) return MOE_ERR_INVALID_ARG;
    n->desc = *d;
    n->device = dev;
    n->num_sms = nsm;
    *out = n;
    return MOE_OK;
}

MOE_API void moe_norm_destroy(moe_norm *n) { free(n); }

MOE_API int moe_add_norm(moe_norm *n, int32_t T, const uint16_t *x, int64_t x_stride,
                         const uint16_t *residual, int64_t residual_stride, uint16_t *total,
                         int64_t total_stride, uint16_t *y, int64_t y_stride, const moe_fp8_rows *y8,
                         void *stream) {
    NvtxRange nvtx_range("moe_add_norm");
    if (!n || T < 0 || (total && !residual)) return MOE_ERR_INVALID_ARG;
    if (T == 0 || (!total && !y && !y8)) return MOE_OK;
    const int d = n->desc.d_model;
    if (!rows_ok(x, x_stride, d) || (residual && !rows_ok(residual, residual_stride, d)) ||
        (total && !rows_ok(total, total_stride, d)) || (y && !rows_ok(y, y_stride, d)) ||
        (y8 && !rows8_ok(y8, d, d % 16 == 8)) || !current(n->device))
        return MOE_ERR_INVALID_ARG;
    MoeNormArgs g = {};
    g.T = T;
    g.d = d;
    g.eps = n->desc.eps;
    g.weight = n->desc.weight;
    g.x = x;
    g.residual = residual;
    g.total = total;
    g.y = y;
    g.x_stride = x_stride;
    g.residual_stride = residual_stride;
    g.total_stride = total_stride;
    g.y_stride = y_stride;
    if (y8) {
        g.q = y8->q;
        g.s = y8->s;
        g.q_stride = y8->q_stride;
        g.s_stride = y8->s_stride;
    }
    return moe_launch_norm(g, n->num_sms, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

MOE_API int moe_linear_create(const moe_linear_desc *d, const uint8_t *w_q, const float *w_s,
                              moe_linear **out) {
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = NULL;
    if (!d || d->d_in <= 0 || d->d_in % 16 || d->d_out <= 0 || d->d_out % 8 || !w_q ||
        !aligned16(w_q) || !w_s || ((uintptr_t)w_s & 3u))
        return MOE_ERR_INVALID_ARG;
    if (d->d_in > 65536 || d->d_out > 1 << 20) return MOE_ERR_UNSUPPORTED;
    int dev = 0, nsm = 0;
    const int rc = check_device(&dev, &nsm);
    if (rc != MOE_OK) return rc;
    if (moe_linear_setup() != cudaSuccess) return MOE_ERR_CUDA;
    moe_linear *l = (moe_linear *)calloc(1, sizeof(moe_linear));
    if (!l) return MOE_ERR_INVALID_ARG;
    l->desc = *d;
    l->w_s = w_s;
    l->device = dev;
    l->num_sms = nsm;
    l->inject = MOE_INJECT_NONE;
    l->timeout = kTimeoutCycles;
    if (!make_map_2d(&l->map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_q, d->d_in, d->d_out, d->d_in, 128,
                     128) ||
        !make_map_2d(&l->map_w64, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_q, d->d_in, d->d_out, d->d_in, 128,
                     64) ||
        cudaMalloc(&l->status, sizeof(int)) != cudaSuccess) {
        free(l);
        return MOE_ERR_CUDA;
    }
    if (cudaMemset(l->status, 0, sizeof(int)) != cudaSuccess) {
        cudaFree(l->status);
        free(l);
        return MOE_ERR_CUDA;
    }
    *out = l;
    return MOE_OK;
}

MOE_API void moe_linear_destroy(moe_linear *l) {
    if (!l) return;
    cudaFree(l->status);
    free(l);
}

MOE_API int moe_linear_forward(moe_linear *l, int32_t T, const moe_fp8_rows *x, void *out,
                               int64_t out_stride, int32_t out_type, void *stream) {
    NvtxRange nvtx_range("moe_linear_forward");
    if (!l || T < 0 || (out_type != MOE_LINEAR_BF16 && out_type != MOE_LINEAR_F32))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const moe_linear_desc &d = l->desc;
    if (!x || !rows8_ok(x, d.d_in) || !out || !aligned16(out) || out_stride < d.d_out ||
        out_stride % (out_type == MOE_LINEAR_F32 ? 4 : 8) || !current(l->device))
        return MOE_ERR_INVALID_ARG;
    if (T > INT32_MAX - 512) return MOE_ERR_UNSUPPORTED;  // 32-bit rows with room for a tile
    MoeLinearArgs g = {};
    g.T = T;
    g.K = d.d_in;
    g.N = d.d_out;
    g.x_s = x->s;
    g.x_s_stride = x->s_stride;
    g.w_s = l->w_s;
    g.out = out;
    g.out_stride = out_stride;
    g.out_f32 = out_type == MOE_LINEAR_F32;
    g.status = l->status;
    g.timeout_cycles = l->timeout;
    g.inject = l->inject;
    const MoeLinearBox box = moe_linear_box(T, d.d_in, d.d_out, l->num_sms);
    CUtensorMap map_x;
    if (!make_map_2d(&map_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, x->q, d.d_in, T, x->q_stride, 128, box.x_rows))
        return MOE_ERR_CUDA;
    return moe_launch_linear(box.w64 ? l->map_w64 : l->map_w, map_x, g, l->num_sms, (cudaStream_t)stream) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

MOE_API int moe_linear_set_fault_injection(moe_linear *l, int32_t mode, int64_t timeout_cycles) {
    if (!l || (mode != MOE_INJECT_NONE && (mode < MOE_INJECT_LINEAR_STALL || mode > MOE_INJECT_LINEAR_STALL_LAST)))
        return MOE_ERR_INVALID_ARG;
    if (timeout_cycles > 0 && timeout_cycles < 100000) return MOE_ERR_INVALID_ARG;
    l->inject = mode;
    l->timeout = timeout_cycles > 0 ? (long long)timeout_cycles : kTimeoutCycles;
    return MOE_OK;
}

MOE_API int moe_linear_status(moe_linear *l, void *stream) {
    if (!l) return MOE_ERR_INVALID_ARG;
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return MOE_ERR_CUDA;
    int v = 0;
    if (cudaMemcpy(&v, l->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (v != 0 && cudaMemset(l->status, 0, sizeof(int)) != cudaSuccess) return MOE_ERR_CUDA;
    return v;
}
