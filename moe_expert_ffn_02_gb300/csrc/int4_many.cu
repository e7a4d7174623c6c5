// The forms of the 4-bit products for many rows: which chunk a call's groups ask for.  Each chunk's kernels are
// compiled in a unit of their own.
#include "experts_internal.cuh"

namespace moe {

cudaError_t launch_int4_many_128(const moe_int4* L, const Int4Call& c, cudaStream_t s);
cudaError_t launch_int4_many_64(const moe_int4* L, const Int4Call& c, cudaStream_t s);
cudaError_t launch_int4_many_32(const moe_int4* L, const Int4Call& c, cudaStream_t s);
double int4_many_us_128(const moe_int4* L, const Int4Call& c);
double int4_many_us_64(const moe_int4* L, const Int4Call& c);
double int4_many_us_32(const moe_int4* L, const Int4Call& c);

namespace {
int chunk_of(const moe_int4* L) { return L->d.group % 128 == 0 || L->groups == 1 ? 128 : L->d.group % 64 == 0 ? 64 : 32; }
}  // namespace

double int4_many_us(const moe_int4* L, const Int4Call& c) {
    const int chunk = chunk_of(L);
    return chunk == 128 ? int4_many_us_128(L, c) : chunk == 64 ? int4_many_us_64(L, c) : int4_many_us_32(L, c);
}

cudaError_t launch_int4_many(const moe_int4* L, const Int4Call& c, cudaStream_t s) {
    const int chunk = chunk_of(L);
    Int4Call call = c;
    call.groups_are_chunks = L->d.group == chunk;
    return chunk == 128 ? launch_int4_many_128(L, call, s) : chunk == 64 ? launch_int4_many_64(L, call, s) : launch_int4_many_32(L, call, s);
}

}  // namespace moe
