// C ABI of the training-side operators (declared in include/orthrus.h):
// argument checks and dispatch; no context, scratch in the caller's
// workspace.
#include "common.cuh"
#include "train.h"

using namespace orthrus;

#define CK(x)                                                                              \
    do {                                                                                   \
        cudaError_t e_ = (x);                                                              \
        if (e_ == cudaErrorNotSupported) return ORTHRUS_ERR_UNSUPPORTED;                   \
        if (e_ != cudaSuccess) return ORTHRUS_ERR_CUDA;                                    \
    } while (0)

namespace {

// the check bits of the calls that name no word of their own, one word per device
__device__ unsigned own_err_word;

__global__ void clear_bits_kernel(unsigned *word, unsigned bits) { atomicAnd(word, ~bits); }

constexpr int32_t kMostRows = 4000000, kMostHidden = 65536;

bool dtype_ok(int32_t t) { return t == ORTHRUS_BF16 || t == ORTHRUS_FP32; }

// a tensor of elements of type t: aligned to its element; NULL only when it is empty
bool ptr_ok(const void *p, int32_t t, bool needed)
{
    if (!p) return !needed;
    return (uintptr_t)p % (t == ORTHRUS_BF16 ? 2 : 4) == 0;
}

orthrus_status_t shape_ok(int32_t rows, int32_t hidden, int32_t vocab)
{
    if (rows < 0 || hidden < 1 || vocab < 1) return ORTHRUS_ERR_INVALID_ARG;
    if (rows > kMostRows || vocab > kMostRows || hidden > kMostHidden) return ORTHRUS_ERR_CAPACITY;
    return ORTHRUS_OK;
}

orthrus_status_t ws_ok(const void *ws, size_t have, size_t need)
{
    if (need == 0) return ORTHRUS_OK;
    if (!ws || (uintptr_t)ws % 256) return ORTHRUS_ERR_INVALID_ARG;
    return have < need ? ORTHRUS_ERR_CAPACITY : ORTHRUS_OK;
}

// where a call of `rows` rows raises its bits
orthrus_status_t err_word(uint32_t *&dev_err, int32_t rows)
{
    if (dev_err || rows == 0) return ORTHRUS_OK;
    void *p = nullptr;
    CK(cudaGetSymbolAddress(&p, own_err_word));
    dev_err = (uint32_t *)p;
    return ORTHRUS_OK;
}

}  // namespace

#define OK(x)                                          \
    do {                                               \
        const orthrus_status_t s_ = (x);               \
        if (s_ != ORTHRUS_OK) return s_;               \
    } while (0)

extern "C" {

orthrus_status_t orthrus_embed_rows(const void *table, int32_t dtype, int32_t vocab, int32_t hidden,
                                    const int32_t *ids, int32_t rows, float scale, void *out, int32_t out_dtype,
                                    uint32_t *dev_err, void *stream)
{
    OK(shape_ok(rows, hidden, vocab));
    if (!dtype_ok(dtype) || !dtype_ok(out_dtype) || !ptr_ok(table, dtype, rows > 0) ||
        !ptr_ok(ids, ORTHRUS_FP32, rows > 0) || !ptr_ok(out, out_dtype, rows > 0) || !ptr_ok(dev_err, ORTHRUS_FP32, false))
        return ORTHRUS_ERR_INVALID_ARG;
    if (rows == 0) return ORTHRUS_OK;
    OK(err_word(dev_err, rows));
    CK(launch_embed_rows(EmbedRowsArgs{table, ids, out, dtype, out_dtype, rows, hidden, vocab, scale, dev_err},
                         (cudaStream_t)stream));
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_embed_grad_workspace(int32_t rows, int32_t hidden, int32_t vocab, size_t *bytes)
{
    if (!bytes) return ORTHRUS_ERR_INVALID_ARG;
    OK(shape_ok(rows, hidden, vocab));
    *bytes = rows ? plan_embed_grad(rows, vocab, hidden).total : 0;
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_embed_grad(const void *dout, int32_t dout_dtype, const int32_t *ids, int32_t rows,
                                    int32_t hidden, int32_t vocab, float scale, int32_t accumulate, void *dtable,
                                    int32_t dtable_dtype, void *workspace, size_t ws_bytes, uint32_t *dev_err,
                                    void *stream)
{
    OK(shape_ok(rows, hidden, vocab));
    if (!dtype_ok(dout_dtype) || !dtype_ok(dtable_dtype) || !ptr_ok(dout, dout_dtype, rows > 0) ||
        !ptr_ok(ids, ORTHRUS_FP32, rows > 0) || !ptr_ok(dtable, dtable_dtype, true) ||
        !ptr_ok(dev_err, ORTHRUS_FP32, false) || (accumulate != 0 && accumulate != 1))
        return ORTHRUS_ERR_INVALID_ARG;
    size_t need;
    OK(orthrus_embed_grad_workspace(rows, hidden, vocab, &need));
    OK(ws_ok(workspace, ws_bytes, need));
    OK(err_word(dev_err, rows));
    CK(launch_embed_grad(EmbedGradArgs{dout, ids, dtable, dout_dtype, dtable_dtype, rows, hidden, vocab, accumulate, scale,
                                       (char *)workspace, dev_err},
                         (cudaStream_t)stream));
    return ORTHRUS_OK;
}

static orthrus_status_t norm_ok(const void *x, int32_t x_dtype, const void *gain, const void *y, int32_t dtype,
                                int32_t rows, int32_t hidden, float eps)
{
    OK(shape_ok(rows, hidden, 1));
    if (!dtype_ok(x_dtype) || !dtype_ok(dtype) || !ptr_ok(x, x_dtype, rows > 0) || !ptr_ok(gain, dtype, rows > 0) ||
        !ptr_ok(y, dtype, rows > 0) || !(eps >= 0.f))
        return ORTHRUS_ERR_INVALID_ARG;
    if (x_dtype == ORTHRUS_BF16 && dtype == ORTHRUS_FP32) return ORTHRUS_ERR_UNSUPPORTED;
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_rmsnorm(const void *x, int32_t x_dtype, const void *gain, int32_t dtype, int32_t rows,
                                 int32_t hidden, float eps, void *y, void *stream)
{
    OK(norm_ok(x, x_dtype, gain, y, dtype, rows, hidden, eps));
    if (rows == 0) return ORTHRUS_OK;
    NormArgs a{};
    a.x = x; a.gain = gain; a.out = y; a.x_dtype = x_dtype; a.dtype = dtype; a.rows = rows; a.d = hidden; a.eps = eps;
    CK(launch_norm_rows(a, (cudaStream_t)stream));
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_rmsnorm_grad_workspace(int32_t rows, int32_t hidden, size_t *bytes)
{
    if (!bytes) return ORTHRUS_ERR_INVALID_ARG;
    OK(shape_ok(rows, hidden, 1));
    *bytes = rows ? norm_grad_workspace(rows, hidden) : 0;
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_rmsnorm_grad(const void *x, int32_t x_dtype, const void *gain, const void *dy, int32_t dtype,
                                      int32_t rows, int32_t hidden, float eps, void *dx, float *dgain,
                                      void *workspace, size_t ws_bytes, void *stream)
{
    OK(norm_ok(x, x_dtype, gain, dy, dtype, rows, hidden, eps));
    if (!ptr_ok(dx, x_dtype, rows > 0) || !ptr_ok(dgain, ORTHRUS_FP32, true)) return ORTHRUS_ERR_INVALID_ARG;
    size_t need;
    OK(orthrus_rmsnorm_grad_workspace(rows, hidden, &need));
    OK(ws_ok(workspace, ws_bytes, need));
    NormArgs a{};
    a.x = x; a.gain = gain; a.dy = dy; a.out = dx; a.dgain = dgain; a.x_dtype = x_dtype; a.dtype = dtype;
    a.rows = rows; a.d = hidden; a.eps = eps; a.ws = (char *)workspace;
    CK(launch_norm_grad(a, (cudaStream_t)stream));
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_ce_lm_head_workspace(int32_t rows, int32_t hidden, int32_t vocab, int32_t dtype, size_t *bytes)
{
    if (!bytes || !dtype_ok(dtype)) return ORTHRUS_ERR_INVALID_ARG;
    OK(shape_ok(rows, hidden, vocab));
    *bytes = rows ? loss_fwd_workspace(rows, hidden, vocab, dtype) : 0;
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_ce_lm_head(const void *h, const void *w, int32_t dtype, const int32_t *targets, int32_t rows,
                                    int32_t hidden, int32_t vocab, float *loss, float *lse, void *workspace,
                                    size_t ws_bytes, uint32_t *dev_err, void *stream)
{
    OK(shape_ok(rows, hidden, vocab));
    const bool some = rows > 0;
    if (!dtype_ok(dtype) || !ptr_ok(h, dtype, some) || !ptr_ok(w, dtype, some) || !ptr_ok(targets, ORTHRUS_FP32, some) ||
        !ptr_ok(loss, ORTHRUS_FP32, some) || !ptr_ok(lse, ORTHRUS_FP32, some) || !ptr_ok(dev_err, ORTHRUS_FP32, false))
        return ORTHRUS_ERR_INVALID_ARG;
    size_t need;
    OK(orthrus_ce_lm_head_workspace(rows, hidden, vocab, dtype, &need));
    OK(ws_ok(workspace, ws_bytes, need));
    OK(err_word(dev_err, rows));
    LossArgs a{};
    a.h = h; a.w = w; a.targets = targets; a.loss = loss; a.lse = lse; a.dtype = dtype; a.N = rows; a.d = hidden;
    a.V = vocab; a.ws = (char *)workspace; a.err = dev_err;
    CK(launch_loss_fwd(a, (cudaStream_t)stream));
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_ce_lm_head_grad_workspace(int32_t rows, int32_t hidden, int32_t vocab, int32_t dtype,
                                                   int32_t weight_grad, size_t *bytes)
{
    if (!bytes || !dtype_ok(dtype) || (weight_grad != 0 && weight_grad != 1)) return ORTHRUS_ERR_INVALID_ARG;
    OK(shape_ok(rows, hidden, vocab));
    *bytes = rows ? loss_grad_workspace(rows, hidden, vocab, dtype, weight_grad, 0) : 0;
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_ce_lm_head_grad(const void *h, const void *w, int32_t dtype, const int32_t *targets,
                                         const float *lse, const float *dloss, int32_t rows, int32_t hidden,
                                         int32_t vocab, void *dh, void *dw, void *workspace, size_t ws_bytes,
                                         uint32_t *dev_err, void *stream)
{
    OK(shape_ok(rows, hidden, vocab));
    const bool some = rows > 0;
    if (!dtype_ok(dtype) || !ptr_ok(h, dtype, some) || !ptr_ok(w, dtype, some) || !ptr_ok(targets, ORTHRUS_FP32, some) ||
        !ptr_ok(lse, ORTHRUS_FP32, some) || !ptr_ok(dloss, ORTHRUS_FP32, some) || !ptr_ok(dh, dtype, some) ||
        !ptr_ok(dw, dtype, false) || !ptr_ok(dev_err, ORTHRUS_FP32, false))
        return ORTHRUS_ERR_INVALID_ARG;
    size_t need;
    OK(orthrus_ce_lm_head_grad_workspace(rows, hidden, vocab, dtype, dw != nullptr, &need));
    OK(ws_ok(workspace, ws_bytes, need));
    OK(err_word(dev_err, rows));
    LossArgs a{};
    a.h = h; a.w = w; a.targets = targets; a.lse_in = lse; a.g = dloss; a.dh = dh; a.dw = dw; a.dtype = dtype;
    a.N = rows; a.d = hidden; a.V = vocab; a.ws = (char *)workspace; a.err = dev_err;
    CK(launch_loss_grad(a, (cudaStream_t)stream));
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_kl_lm_head_grad_workspace(int32_t rows, int32_t hidden, int32_t vocab, int32_t dtype,
                                                   size_t *bytes)
{
    if (!bytes || !dtype_ok(dtype)) return ORTHRUS_ERR_INVALID_ARG;
    OK(shape_ok(rows, hidden, vocab));
    *bytes = rows ? loss_grad_workspace(rows, hidden, vocab, dtype, 0, 1) : 0;
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_kl_lm_head_grad(const void *h_ar, const void *h_diff, const void *w, int32_t dtype,
                                         const float *lse_ar, const float *lse_diff, const float *dkl, int32_t rows,
                                         int32_t hidden, int32_t vocab, void *dh_diff, void *workspace,
                                         size_t ws_bytes, uint32_t *dev_err, void *stream)
{
    OK(shape_ok(rows, hidden, vocab));
    const bool some = rows > 0;
    if (!dtype_ok(dtype) || !ptr_ok(h_ar, dtype, some) || !ptr_ok(h_diff, dtype, some) || !ptr_ok(w, dtype, some) ||
        !ptr_ok(lse_ar, ORTHRUS_FP32, some) || !ptr_ok(lse_diff, ORTHRUS_FP32, some) || !ptr_ok(dkl, ORTHRUS_FP32, some) ||
        !ptr_ok(dh_diff, dtype, some) || !ptr_ok(dev_err, ORTHRUS_FP32, false))
        return ORTHRUS_ERR_INVALID_ARG;
    if (rows == 0) return ORTHRUS_OK;
    size_t need;
    OK(orthrus_kl_lm_head_grad_workspace(rows, hidden, vocab, dtype, &need));
    OK(ws_ok(workspace, ws_bytes, need));
    OK(err_word(dev_err, rows));
    LossArgs a{};
    a.h = h_ar; a.h2 = h_diff; a.w = w; a.lse_in = lse_ar; a.lse2_in = lse_diff; a.g = dkl; a.dh = dh_diff;
    a.dtype = dtype; a.N = rows; a.d = hidden; a.V = vocab; a.kl = 1; a.ws = (char *)workspace; a.err = dev_err;
    CK(launch_loss_grad(a, (cudaStream_t)stream));
    return ORTHRUS_OK;
}

orthrus_status_t orthrus_train_check_error(void *stream, uint32_t *bits)
{
    if (!bits) return ORTHRUS_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    void *p = nullptr;
    unsigned h = 0;
    CK(cudaGetSymbolAddress(&p, own_err_word));
    CK(cudaMemcpyAsync(&h, p, 4, cudaMemcpyDeviceToHost, s));
    CK(cudaStreamSynchronize(s));
    if (h) {   // (only what is reported: another stream may raise more meanwhile)
        clear_bits_kernel<<<1, 1, 0, s>>>((unsigned *)p, h);
        CK(cudaGetLastError());
        CK(cudaStreamSynchronize(s));
    }
    *bits = h;
    if (h & ORTHRUS_DEVERR_NONFINITE) return ORTHRUS_ERR_NONFINITE;
    return h ? ORTHRUS_ERR_DEVICE_CHECK : ORTHRUS_OK;
}

}  // extern "C"
