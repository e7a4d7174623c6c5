// 4-bit products, many rows, groups of an odd multiple of 32 channels (int4_many.cuh).
#include "int4_many.cuh"

namespace moe {

cudaError_t launch_int4_many_32(const moe_int4* L, const Int4Call& c, cudaStream_t s) { return launch_mode<4>(L, c, s); }
double int4_many_us_32(const moe_int4* L, const Int4Call& c) { return many_us<4>(L, c); }

}  // namespace moe
