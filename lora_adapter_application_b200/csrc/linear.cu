// Entry points of the dense products (contracts: lora_linear and
// lora_expert_linear in lora_delta.h): the checks, and the kernel for a call.
#include "linear.cuh"

namespace lora {

namespace {

// What both entry points ask of their operands; fills the shared part of `a`.
int check_dense(LinArgs &a, const lora_epilogue *ep, lora_dtype dtype) {
    if (dtype != LORA_BF16 && dtype != LORA_FP32) return LORA_ERR_DTYPE;
    lora_epilogue none{};
    if (!ep) ep = &none;
    if (ep->act < LORA_ACT_NONE || ep->act > LORA_ACT_RELU) return LORA_ERR_SHAPE;
    if (a.d_in < 1 || a.d_in > LORA_MX_MAX || a.d_out < 1 || a.d_out > LORA_MX_MAX / (ep->gated ? 2 : 1)) return LORA_ERR_SHAPE;
    a.n_w = ep->gated ? 2 * a.d_out : a.d_out;
    a.bias = ep->bias, a.addend = ep->addend, a.residual = ep->residual;
    a.ld_a = ep->ld_addend, a.ld_r = ep->ld_residual, a.act = ep->act;
    if (a.ld_x < a.d_in || a.ld_w < a.d_in || a.ld_y < a.d_out || (a.addend && a.ld_a < a.n_w) || (a.residual && a.ld_r < a.d_out))
        return LORA_ERR_SHAPE;
    if (!a.status) return LORA_ERR_NULL;
    if (a.T == 0) return LORA_OK;
    if (!a.y || !a.x || !a.w) return LORA_ERR_NULL;
    const uintptr_t es = dtype == LORA_BF16 ? 2 : 4;
    for (const void *p : {static_cast<const void *>(a.y), a.x, a.w, a.bias, a.addend, a.residual})
        if (!mx_aligned(p, es)) return LORA_ERR_ALIGN;   // no access of an element reaches those
    for (const int32_t *p : {static_cast<const int32_t *>(a.status), a.perm, a.seg_start})
        if (!mx_aligned(p, 4)) return LORA_ERR_ALIGN;
    // in place over the residual, or over the addend where its columns are y's
    if (a.y == a.x || (a.y == a.residual && a.ld_y != a.ld_r) || (a.y == a.addend && (ep->gated || a.ld_y != a.ld_a)))
        return LORA_ERR_SHAPE;
    return LORA_OK;
}

int launch_dense(const LinArgs &a, int64_t x_rows, bool gated, lora_dtype dtype, cudaStream_t st) {
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_rc(e);
    return dtype == LORA_BF16 ? launch_linear_tc(a, x_rows, gated, dev, st) : launch_linear_simt(a, gated, sms, st);
}

}  // namespace

}  // namespace lora

extern "C" {

int lora_linear(void *y, int64_t ld_y, const void *x, int64_t ld_x, const void *w, int64_t ld_w, int32_t T, int32_t d_in,
                int32_t d_out, const lora_epilogue *ep, lora_dtype dtype, int32_t *status, void *stream) {
    using namespace lora;
    if (T < 0 || T > LORA_MAX_ROWS) return LORA_ERR_SHAPE;
    LinArgs a{};
    a.y = y, a.ld_y = ld_y, a.x = x, a.ld_x = ld_x, a.w = w, a.ld_w = ld_w;
    a.T = T, a.d_in = d_in, a.d_out = d_out, a.status = status, a.N = 1, a.x_div = 1;
    const int rc = check_dense(a, ep, dtype);
    if (rc != LORA_OK || T == 0) return rc;
    return launch_dense(a, T, ep && ep->gated, dtype, static_cast<cudaStream_t>(stream));
}

int lora_expert_linear(void *y, int64_t ld_y, const void *x, int64_t ld_x, int32_t x_rows, int32_t x_div, const void *w,
                       int32_t d_in, int32_t d_out, const lora_meta *meta, const lora_epilogue *ep, lora_dtype dtype,
                       int32_t *status, void *stream) {
    using namespace lora;
    int rc = check_meta_args(meta);
    if (rc != LORA_OK) return rc;
    if (meta->N > LORA_MAX_EXPERTS || x_div < 1 || x_rows < 0 || ((int64_t)meta->T + x_div - 1) / x_div > x_rows) return LORA_ERR_SHAPE;
    LinArgs a{};
    a.y = y, a.ld_y = ld_y, a.x = x, a.ld_x = ld_x, a.w = w, a.ld_w = d_in;
    a.T = meta->T, a.d_in = d_in, a.d_out = d_out, a.status = status;
    a.perm = meta->perm, a.seg_start = meta->seg_start, a.N = meta->N, a.x_div = x_div;
    rc = check_dense(a, ep, dtype);
    if (rc != LORA_OK || a.T == 0) return rc;
    return launch_dense(a, x_rows, ep && ep->gated, dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
