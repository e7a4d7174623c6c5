// C ABI of the operators around experts outside the fused layer (declared in
// include/moe.h): argument checks and launches.
#include "api_common.cuh"
#include "experts_internal.cuh"

using moe::aligned;
using moe::cuda_fail;
using moe::fail;
using moe::read_status;

namespace {

moe_status check_type(int type, const char* what) {
    return type == MOE_BF16 || type == MOE_F32 ? MOE_OK : fail(MOE_ERR_INVALID_ARG, "unknown %s type %d", what, type);
}

// Counts shared by the three calls.
moe_status check_pairs(int tokens, int top_k) {
    if (tokens < 0 || top_k < 1) return fail(MOE_ERR_INVALID_ARG, "tokens = %d, top_k = %d", tokens, top_k);
    if (top_k > MOE_DISPATCH_MAX_TOPK) return fail(MOE_ERR_UNSUPPORTED, "top_k (%d) is over %d", top_k, MOE_DISPATCH_MAX_TOPK);
    // a grid has a block more than there are tokens, or 65535 planes of 32768
    if ((int64_t)tokens * top_k > MOE_DISPATCH_MAX_PAIRS)
        return fail(MOE_ERR_UNSUPPORTED, "tokens * top_k is over %d", MOE_DISPATCH_MAX_PAIRS);
    return MOE_OK;
}

moe_status check_cols(int cols, int n_rows) {
    if (cols < 1 || n_rows < 0) return fail(MOE_ERR_INVALID_ARG, "cols = %d, n_rows = %d", cols, n_rows);
    if (cols > MOE_DISPATCH_MAX_COLS) return fail(MOE_ERR_UNSUPPORTED, "cols (%d) is over %d", cols, MOE_DISPATCH_MAX_COLS);
    return MOE_OK;
}

// One matrix operand: elements on their own boundaries, rows that do not overlap.
moe_status check_rows(const void* p, int64_t ld, int type, int cols, const char* what) {
    if (!p) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", what);
    if (!aligned(p, type == MOE_F32 ? 4 : 2)) return fail(MOE_ERR_INVALID_ARG, "%s is not aligned to its elements", what);
    if (ld < cols) return fail(MOE_ERR_INVALID_ARG, "%s: a row stride (%lld) is less than cols (%d)", what, (long long)ld, cols);
    return MOE_OK;
}

moe_status check_words(const void* p, const char* what) {
    return p && aligned(p, 4) ? MOE_OK : fail(MOE_ERR_INVALID_ARG, "%s is NULL or not 4-byte aligned", what);
}

}  // namespace

MOE_EXPORT moe_status moe_dispatch_workspace_bytes(int32_t tokens, int32_t top_k, int32_t n_experts, size_t* bytes) {
    if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    moe_status st = check_pairs(tokens, top_k);
    if (st != MOE_OK) return st;
    if (n_experts < 1) return fail(MOE_ERR_INVALID_ARG, "n_experts = %d", n_experts);
    if (n_experts > MOE_DISPATCH_MAX_EXPERTS)
        return fail(MOE_ERR_UNSUPPORTED, "n_experts (%d) is over %d", n_experts, MOE_DISPATCH_MAX_EXPERTS);
    const moe::SortPlan plan = moe::plan_sort(tokens, top_k);
    if (plan.chunks) *bytes = ((size_t)(plan.most_chunks + 1) * n_experts * sizeof(int32_t) + 255) / 256 * 256;
    return MOE_OK;
}

MOE_EXPORT moe_status moe_dispatch(const moe_dispatch_args* a, void* ws, size_t ws_bytes, void* stream) {
    if (!a) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    size_t need = 0;
    moe_status st = moe_dispatch_workspace_bytes(a->tokens, a->top_k, a->n_experts, &need);
    if (st != MOE_OK) return st;
    if (a->first_expert < 0 || a->first_expert > INT32_MAX - a->n_experts)
        return fail(MOE_ERR_INVALID_ARG, "first_expert = %d", a->first_expert);
    if (!a->ids && !a->x) return fail(MOE_ERR_INVALID_ARG, "neither ids to sort nor x to copy");
    if (a->x) {
        st = check_type(a->x_type, "x");
        if (st == MOE_OK) st = check_cols(a->cols, a->n_rows);
        if (st == MOE_OK && a->tokens > 0) st = check_rows(a->x, a->ldx, a->x_type, a->cols, "x");
        if (st == MOE_OK && a->tokens > 0 && a->n_rows > 0) st = check_rows(a->rows, a->ld_rows, a->x_type, a->cols, "rows");
        if (st != MOE_OK) return st;
    }
    if (a->ids) {
        st = check_words(a->expert_offsets, "expert_offsets");
        if (st == MOE_OK && a->tokens > 0) st = check_words(a->ids, "ids");
        if (st == MOE_OK && a->tokens > 0) st = check_words(a->sorted_token, "sorted_token");
    }
    if (st == MOE_OK && a->tokens > 0) st = check_words(a->inv_row, "inv_row");
    if (st != MOE_OK) return st;
    if (a->ids && need) {
        if (!ws || !aligned(ws, 256)) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
        if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, %zu are needed", ws_bytes, need);
    }
    if (!a->ids && a->tokens == 0) return MOE_OK;
    cudaError_t e = moe::launch_dispatch(a, static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "dispatch");
}

MOE_EXPORT moe_status moe_combine(const moe_combine_args* a, void* stream) {
    if (!a) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    moe_status st = check_pairs(a->tokens, a->top_k);
    if (st == MOE_OK) st = check_cols(a->cols, a->n_rows);
    if (st == MOE_OK) st = check_type(a->o_type, "o");
    if (st == MOE_OK) st = check_type(a->y_type, "y");
    if (st != MOE_OK || a->tokens == 0) return st;
    st = check_words(a->inv_row, "inv_row");
    if (st == MOE_OK && a->w) st = check_words(a->w, "w");
    if (st == MOE_OK && a->n_rows > 0) st = check_rows(a->o, a->ldo, a->o_type, a->cols, "o");
    if (st == MOE_OK && a->add) st = check_rows(a->add, a->ld_add, a->y_type, a->cols, "add");
    if (st == MOE_OK) st = check_rows(a->y, a->ldy, a->y_type, a->cols, "y");
    if (st != MOE_OK) return st;
    cudaError_t e = moe::launch_combine_rows(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "combine");
}

MOE_EXPORT moe_status moe_combine_grad(const moe_combine_grad_args* a, void* stream) {
    if (!a) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    moe_status st = check_pairs(a->tokens, a->top_k);
    if (st == MOE_OK) st = check_cols(a->cols, a->n_rows);
    if (st == MOE_OK) st = check_type(a->o_type, "o");
    if (st == MOE_OK) st = check_type(a->y_type, "y");
    if (st != MOE_OK || a->tokens == 0) return st;
    if (!a->d_o && !a->d_w && a->n_rows > 0) return fail(MOE_ERR_INVALID_ARG, "no output");
    st = check_words(a->inv_row, "inv_row");
    if (st == MOE_OK && a->w) st = check_words(a->w, "w");
    if (st == MOE_OK) st = check_rows(a->dy, a->ld_dy, a->y_type, a->cols, "dy");
    if (st == MOE_OK && a->d_w) st = check_words(a->d_w, "d_w");
    if (st == MOE_OK && a->d_w && a->n_rows > 0) st = check_rows(a->o, a->ldo, a->o_type, a->cols, "o");
    if (st == MOE_OK && a->d_o && a->n_rows > 0) st = check_rows(a->d_o, a->ld_d_o, a->o_type, a->cols, "d_o");
    if (st != MOE_OK) return st;
    cudaError_t e = moe::launch_combine_grad(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "combine gradient");
}

MOE_EXPORT moe_status moe_dispatch_device_status(void* stream, uint32_t* flags) {
    uint32_t* word = nullptr;
    cudaError_t e = moe::dispatch_status_word(&word);
    return e != cudaSuccess ? cuda_fail(e, "the dispatch's status word") : read_status(word, stream, flags);
}
