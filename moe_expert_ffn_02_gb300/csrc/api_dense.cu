// C ABI of the dense operators (declared in include/moe.h): argument checks,
// weight ownership and launches.
#include "api_common.cuh"
#include "dense_internal.cuh"

#include <climits>
#include <new>

using moe::aligned;
using moe::cuda_fail;
using moe::fail;
using moe::kDefaultWaitLimitUs;
using moe::read_status;

namespace {

moe_status check_fp8(const moe_fp8_matrix& m, int rows, int cols, const char* what) {
    if (!m.q || !m.s) return fail(MOE_ERR_INVALID_ARG, "%s: codes or scales are NULL", what);
    if (!aligned(m.q, 16) || m.ldq % 16) return fail(MOE_ERR_INVALID_ARG, "%s: code rows are not on 16-byte strides", what);
    if (m.ldq < cols) return fail(MOE_ERR_INVALID_ARG, "%s: ldq (%lld) is less than the %d columns", what, (long long)m.ldq, cols);
    if (m.lds < rows) return fail(MOE_ERR_INVALID_ARG, "%s: lds (%lld) is less than the %d rows", what, (long long)m.lds, rows);
    if (m.scale_type != MOE_SCALE_F32 && m.scale_type != MOE_SCALE_E8M0)
        return fail(MOE_ERR_INVALID_ARG, "%s: unknown scale type %d", what, m.scale_type);
    if (!aligned(m.s, 16) || m.lds % (m.scale_type == MOE_SCALE_F32 ? 4 : 16))
        return fail(MOE_ERR_INVALID_ARG, "%s: scale rows are not on 16-byte strides", what);
    return MOE_OK;
}

moe_status check_linear(const moe_linear* L) {
    if (!L) return fail(MOE_ERR_INVALID_ARG, "linear is NULL");
    int cur = -1;
    cudaError_t e = cudaGetDevice(&cur);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (cur != L->device)
        return fail(MOE_ERR_INVALID_ARG, "the current device (%d) is not the weights' device (%d)", cur, L->device);
    return MOE_OK;
}

moe_status check_input(const moe_linear* L, const moe_fp8_matrix* a, int rows) {
    if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows = %d is negative", rows);
    if (rows > MOE_LINEAR_MAX_ROWS) return fail(MOE_ERR_UNSUPPORTED, "rows (%d) is over %d", rows, MOE_LINEAR_MAX_ROWS);
    if (!a) return fail(MOE_ERR_INVALID_ARG, "a is NULL");
    if (rows == 0) return MOE_OK;
    moe_status st = check_fp8(*a, rows, L->d.in_features, "a");
    if (st != MOE_OK) return st;
    if (a->scale_type != L->d.scale_type)
        return fail(MOE_ERR_INVALID_ARG, "a's scale type (%d) is not the weights' (%d)", a->scale_type, L->d.scale_type);
    return MOE_OK;
}

}  // namespace

MOE_EXPORT moe_status moe_add_rmsnorm(const moe_rmsnorm_args* a, void* stream) {
    if (!a) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    if (a->rows < 0 || a->cols < 1) return fail(MOE_ERR_INVALID_ARG, "rows = %d, cols = %d", a->rows, a->cols);
    if (a->cols > MOE_RMSNORM_MAX_COLS)
        return fail(MOE_ERR_UNSUPPORTED, "cols (%d) is over %d", a->cols, MOE_RMSNORM_MAX_COLS);
    if (a->x_type != MOE_BF16 && a->x_type != MOE_F32) return fail(MOE_ERR_INVALID_ARG, "unknown x type %d", a->x_type);
    if (a->res_type != MOE_BF16 && a->res_type != MOE_F32)
        return fail(MOE_ERR_INVALID_ARG, "unknown residual type %d", a->res_type);
    if (a->res && a->x_type == MOE_F32 && a->res_type == MOE_BF16)
        return fail(MOE_ERR_UNSUPPORTED, "an fp32 x with a bf16 residual stream");
    if (!(a->eps >= 0.0f)) return fail(MOE_ERR_INVALID_ARG, "eps must be at least 0");
    if (a->rows == 0) return MOE_OK;
    if (!a->x || !a->weight) return fail(MOE_ERR_INVALID_ARG, "x or weight is NULL");
    if (a->res_out && !a->res) return fail(MOE_ERR_INVALID_ARG, "res_out without a residual");
    if (!a->y && !a->out.q && !a->res_out) return fail(MOE_ERR_INVALID_ARG, "no output");
    const size_t xs = a->x_type == MOE_F32 ? 4 : 2, rs = a->res_type == MOE_F32 ? 4 : 2;
    if (!aligned(a->x, xs) || !aligned(a->y, xs) || !aligned(a->res, rs) || !aligned(a->res_out, rs) ||
        !aligned(a->weight, 4))
        return fail(MOE_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    if (a->ldx < a->cols || (a->res && a->ld_res < a->cols) || (a->res_out && a->ld_res_out < a->cols) ||
        (a->y && a->ldy < a->cols))
        return fail(MOE_ERR_INVALID_ARG, "a row stride is less than cols (%d)", a->cols);
    if (a->out.q || a->out.s) {
        moe_status st = check_fp8(a->out, a->rows, a->cols, "out");
        if (st != MOE_OK) return st;
    }
    cudaError_t e = moe::launch_rmsnorm(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "residual RMS norm");
}

MOE_EXPORT moe_status moe_linear_create(const moe_linear_desc* d, const moe_linear_weights* w, void* stream,
                                        moe_linear** out) {
    if (!d || !w || !out) return fail(MOE_ERR_INVALID_ARG, "desc, weights and out must be non-NULL");
    *out = nullptr;
    if (d->in_features < 1 || d->out_features < 1 || d->in_features > MOE_LINEAR_MAX_FEATURES ||
        d->out_features > MOE_LINEAR_MAX_FEATURES)
        return fail(MOE_ERR_UNSUPPORTED, "in_features (%d) and out_features (%d) must lie in [1, %d]", d->in_features,
                    d->out_features, MOE_LINEAR_MAX_FEATURES);
    if (d->gated != 0 && d->gated != 1) return fail(MOE_ERR_INVALID_ARG, "gated must be 0 or 1");
    if (d->scale_type != MOE_SCALE_F32 && d->scale_type != MOE_SCALE_E8M0)
        return fail(MOE_ERR_INVALID_ARG, "unknown scale type %d", d->scale_type);
    if (!w->w || !w->s || (d->gated && (!w->w_up || !w->s_up)))
        return fail(MOE_ERR_INVALID_ARG, "a weight or scale pointer is NULL");
    if (d->scale_type == MOE_SCALE_F32 && (!aligned(w->s, 4) || (d->gated && !aligned(w->s_up, 4))))
        return fail(MOE_ERR_INVALID_ARG, "scales are not 4-byte aligned");
    moe_linear* L = new (std::nothrow) moe_linear{};
    if (!L) return fail(MOE_ERR_CUDA, "out of host memory");
    L->d = *d;
    L->wait_limit = kDefaultWaitLimitUs;
    L->kt = (d->in_features + moe::QB - 1) / moe::QB;
    L->rows = d->gated ? 2 * ((d->out_features + 7) / 8 * 8) : d->out_features;
    L->rows_pad = (L->rows + 7) / 8 * 8;
    const size_t nsw = (size_t)(d->gated ? 2 : 1) * ((d->out_features + moe::QB - 1) / moe::QB) * L->kt;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const char* what = "device query";
    cudaError_t e = cudaGetDevice(&L->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&L->num_sms, cudaDevAttrMultiProcessorCount, L->device);
    if (e == cudaSuccess) moe::plan_fp8_few(L);
    if (e == cudaSuccess) what = "allocating weights", e = cudaMalloc(&L->w, (size_t)L->kt * L->rows_pad * 128);
    if (e == cudaSuccess) what = "allocating scales", e = cudaMalloc(&L->sw, nsw * 4);
    if (e == cudaSuccess && d->scale_type == MOE_SCALE_E8M0)
        what = "allocating scale factors", e = cudaMalloc(&L->wsf, (size_t)((L->kt + 3) / 4) * ((L->rows_pad + moe::QB - 1) / moe::QB) * 512);
    if (e == cudaSuccess) what = "allocating status", e = cudaMalloc(&L->dev_status, 4);
    if (e == cudaSuccess) what = "memset", e = cudaMemsetAsync(L->dev_status, 0, 4, s);
    if (e == cudaSuccess)
        what = "weight repack", e = moe::launch_linear_repack(L, w->w, w->s, d->gated ? w->w_up : nullptr,
                                                              d->gated ? w->s_up : nullptr, s);
    if (e == cudaSuccess) what = "moe_linear_create synchronise", e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) {
        moe_status st = cuda_fail(e, what);
        cudaFree(L->w); cudaFree(L->sw); cudaFree(L->wsf); cudaFree(L->dev_status);
        delete L;
        return st;
    }
    *out = L;
    return MOE_OK;
}

MOE_EXPORT moe_status moe_linear_destroy(moe_linear* L) {
    if (!L) return fail(MOE_ERR_INVALID_ARG, "linear is NULL");
    int cur = -1;
    cudaError_t e = cudaGetDevice(&cur);
    if (e == cudaSuccess && cur != L->device) e = cudaSetDevice(L->device);
    if (e != cudaSuccess) return cuda_fail(e, "moe_linear_destroy: selecting the weights' device");
    e = cudaDeviceSynchronize();
    cudaFree(L->w); cudaFree(L->sw); cudaFree(L->wsf); cudaFree(L->dev_status);
    const int dev = L->device;
    delete L;
    if (cur >= 0 && cur != dev) cudaSetDevice(cur);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_linear_destroy synchronise");
}

MOE_EXPORT moe_status moe_linear_forward(moe_linear* L, const moe_fp8_matrix* a, int32_t rows, void* y, int64_t ldy,
                                         int32_t y_type, void* stream) {
    moe_status st = check_linear(L);
    if (st == MOE_OK && L->d.gated) st = fail(MOE_ERR_INVALID_ARG, "gated weights: call moe_gated_linear_forward");
    if (st == MOE_OK) st = check_input(L, a, rows);
    if (st != MOE_OK) return st;
    if (y_type != MOE_BF16 && y_type != MOE_F32) return fail(MOE_ERR_INVALID_ARG, "unknown y type %d", y_type);
    if (rows == 0) return MOE_OK;
    if (!y || !aligned(y, y_type == MOE_F32 ? 4 : 2)) return fail(MOE_ERR_INVALID_ARG, "y is NULL or misaligned");
    if (ldy < L->d.out_features)
        return fail(MOE_ERR_INVALID_ARG, "ldy (%lld) is less than out_features (%d)", (long long)ldy, L->d.out_features);
    moe::GemmCall c = {};
    c.lin = L;
    c.plant = L->plant.load(std::memory_order_relaxed) && L->plant.exchange(false);     // threads may share the weights
    c.aq = a->q; c.ld_aq = a->ldq; c.as = a->s; c.ld_as = a->lds;
    c.M = rows;
    c.y = y; c.ldy = ldy; c.y_f32 = y_type == MOE_F32;
    cudaError_t e = moe::launch_fp8_linear(c, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "FP8 linear");
}

MOE_EXPORT moe_status moe_gated_linear_forward(moe_linear* L, const moe_fp8_matrix* a, int32_t rows,
                                               const moe_fp8_matrix* h, void* stream) {
    moe_status st = check_linear(L);
    if (st == MOE_OK && !L->d.gated) st = fail(MOE_ERR_INVALID_ARG, "plain weights: call moe_linear_forward");
    if (st == MOE_OK) st = check_input(L, a, rows);
    if (st != MOE_OK) return st;
    if (!h) return fail(MOE_ERR_INVALID_ARG, "h is NULL");
    if (rows == 0) return MOE_OK;
    st = check_fp8(*h, rows, L->d.out_features, "h");
    if (st != MOE_OK) return st;
    if (h->scale_type != L->d.scale_type)
        return fail(MOE_ERR_INVALID_ARG, "h's scale type (%d) is not the weights' (%d)", h->scale_type, L->d.scale_type);
    moe::GemmCall c = {};
    c.lin = L;
    c.plant = L->plant.load(std::memory_order_relaxed) && L->plant.exchange(false);     // threads may share the weights
    c.aq = a->q; c.ld_aq = a->ldq; c.as = a->s; c.ld_as = a->lds;
    c.M = rows;
    c.hq = h->q; c.ld_hq = h->ldq; c.hs = h->s; c.ld_hs = h->lds;
    cudaError_t e = moe::launch_fp8_gated(c, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "FP8 gated linear");
}

MOE_EXPORT moe_status moe_linear_device_status(moe_linear* L, void* stream, uint32_t* flags) {
    moe_status st = check_linear(L);
    return st != MOE_OK ? st : read_status(L->dev_status, stream, flags);
}

MOE_EXPORT moe_status moe_linear_set_wait_limit(moe_linear* L, uint32_t microseconds) {
    if (!L) return fail(MOE_ERR_INVALID_ARG, "linear is NULL");
    if (microseconds == 0) return fail(MOE_ERR_INVALID_ARG, "limit must be positive");
    L->wait_limit = microseconds;
    return MOE_OK;
}

MOE_EXPORT moe_status moe_linear_debug_timeout(moe_linear* L) {
    if (!L) return fail(MOE_ERR_INVALID_ARG, "linear is NULL");
    L->plant = true;
    return MOE_OK;
}

MOE_EXPORT moe_status moe_rmsnorm_device_status(void* stream, uint32_t* flags) {
    uint32_t* word = nullptr;
    cudaError_t e = moe::norm_status_word(&word);
    return e != cudaSuccess ? cuda_fail(e, "the norm's status word") : read_status(word, stream, flags);
}

MOE_EXPORT moe_status moe_rmsnorm_set_wait_limit(uint32_t microseconds) {
    if (microseconds == 0) return fail(MOE_ERR_INVALID_ARG, "limit must be positive");
    moe::norm_set_wait_limit(microseconds);
    return MOE_OK;
}

MOE_EXPORT moe_status moe_rmsnorm_debug_timeout(void) {
    moe::norm_plant_timeout();
    return MOE_OK;
}
