// Internal definitions of the operators that run experts outside the fused
// layer: dispatch and combine with their gradients, products with 4-bit
// weights.  Nothing here is part of the public ABI.
#pragma once
#include "moe_internal.cuh"

namespace moe {

// Tokens per chunk of the multi-CTA sort and the chunks of a call, and no fewer than any smaller batch has
// (the workspace, int32 [most_chunks + 1][n_experts]).  chunks = 0: one kernel does it without workspace.
struct SortPlan {
    int chunk_tokens, chunks, most_chunks;
};
SortPlan plan_sort(int tokens, int top_k);

cudaError_t launch_dispatch(const moe_dispatch_args* a, int32_t* ws, cudaStream_t s);
cudaError_t launch_combine_rows(const moe_combine_args* a, cudaStream_t s);
cudaError_t launch_combine_grad(const moe_combine_grad_args* a, cudaStream_t s);
cudaError_t dispatch_status_word(uint32_t** p);         // the current device's

}  // namespace moe
