// 4-bit products, many rows, groups of whole 128 channels, or one scale per row (int4_many.cuh).
#include "int4_many.cuh"

namespace moe {

cudaError_t launch_int4_many_128(const moe_int4* L, const Int4Call& c, cudaStream_t s) { return launch_mode<1>(L, c, s); }
double int4_many_us_128(const moe_int4* L, const Int4Call& c) { return many_us<1>(L, c); }

}  // namespace moe
