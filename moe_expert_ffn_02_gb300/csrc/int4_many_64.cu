// 4-bit products, many rows, groups of an odd multiple of 64 channels (int4_many.cuh).
#include "int4_many.cuh"

namespace moe {

cudaError_t launch_int4_many_64(const moe_int4* L, const Int4Call& c, cudaStream_t s) { return launch_mode<2>(L, c, s); }
double int4_many_us_64(const moe_int4* L, const Int4Call& c) { return many_us<2>(L, c); }

}  // namespace moe
