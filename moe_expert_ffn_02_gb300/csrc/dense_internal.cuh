// Internal definitions of the dense operators (residual RMS norm, FP8 linear
// and gated projections).  Nothing here is part of the public ABI.
#pragma once
#include <cuda.h>

#include <atomic>

#include "moe_internal.cuh"

struct moe_linear {
    moe_linear_desc d;
    int device;
    int num_sms;
    int rows;              // weight-image rows in use: N, or 2 * up(N, 8) when gated
    int rows_pad;          // rows per K block of the image (multiple of 8)
    int kt;                // K blocks: ceil(K / 128)
    uint8_t* w;            // [kt][rows_pad][128 B] E4M3, 128-byte swizzle, zeros past N and K
    float* sw;             // [1 or 2][ceil(N / 128)][kt] weight scales (gated: gate, then up)
    uint8_t* wsf;          // e8m0: [ceil(kt / 4)][ceil(rows_pad / 128)][512 B] scale-factor blocks of the image's rows
    uint32_t* dev_status;  // device status word
    uint32_t wait_limit;
    std::atomic<bool> plant;  // moe_linear_debug_timeout, for the next forward call
    int few_R, few_S, few_G;  // the few-token form's rows per tile, K ranges and K blocks per stage; few_R 0: it does not fit
};

namespace moe {

// Limit of the waits that let a CTA's own copies and MMAs finish before it leaves, whatever the limit of the
// others: leaving earlier would let them land in memory that is no longer its own.
constexpr uint32_t LANDING_LIMIT_US = 2000000u;

// Scale of a quantisation group from its largest magnitude, shared by the
// norm and the gated projection.  f32: amax / 448.  e8m0: the smallest power
// of two that is at least amax / 448, held as its biased exponent; found from
// the rounded quotient's bits (a non-zero mantissa rounds the exponent up).  A
// group whose quotient lies below the normal range (2^-126) gets scale 1, so
// 1 / s is finite and its codes are zeros.  NaN and infinity give a NaN (e8m0:
// code 255) or infinite scale: they are not hidden.  (With an infinite scale, 1 / s
// is 0: finite values get code 0, infinite ones NaN.)
// `held` is what the scale array stores (the float's bits, or the byte).
__device__ __forceinline__ float group_scale(float amax, bool e8m0, uint32_t& held) {
    float s = __fdiv_rn(amax, 448.0f);
    if (s < 1.17549435e-38f) s = 1.0f;
    if (!e8m0) {
        held = __float_as_uint(s);
        return s;
    }
    const uint32_t b = __float_as_uint(s);
    uint32_t ex = (b >> 23) + ((b & 0x7FFFFFu) ? 1u : 0u);
    if (ex > 254u) ex = 255u;                       // infinity or NaN
    held = ex;
    return __uint_as_float(ex == 255u ? 0x7FC00000u : ex << 23);
}

// 1 / s for the scales above: finite scales lie in [2^-126, 2^120].
__device__ __forceinline__ float inv_scale(float s) { return __frcp_rn(s); }

// 2^(b - 127): the exponent field as it is, except 0 (a subnormal) and 255 (NaN), which both need
// the mantissa's top bit.
__device__ __forceinline__ float e8m0_to_f32(uint8_t b) {
    return __uint_as_float(((uint32_t)b << 23) | ((uint8_t)(b + 1) <= 1 ? 0x400000u : 0u));
}

// max that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Arguments of one GEMM call (plain: y; gated: codes and scales).
struct GemmCall {
    const moe_linear* lin;
    const uint8_t* aq;
    int64_t ld_aq;
    const void* as;
    int64_t ld_as;
    int M;
    void* y;               // plain
    int64_t ldy;
    bool y_f32;
    uint8_t* hq;           // gated
    int64_t ld_hq;
    void* hs;
    int64_t ld_hs;
    bool plant;
};

cudaError_t launch_rmsnorm(const moe_rmsnorm_args* a, cudaStream_t s);
cudaError_t norm_status_word(uint32_t** p);             // the current device's
void norm_set_wait_limit(uint32_t us);
void norm_plant_timeout();
cudaError_t launch_linear_repack(const moe_linear* L, const uint8_t* w, const void* s, const uint8_t* wu,
                                 const void* su, cudaStream_t st);
cudaError_t launch_fp8_linear(const GemmCall& c, cudaStream_t s);
cudaError_t launch_fp8_gated(const GemmCall& c, cudaStream_t s);
struct MxPlan {
    int bn, S;             // rows per tile, K ranges; bn 0: the form does not take these weights
    double us;             // estimate
};
MxPlan plan_fp8_mx(const GemmCall& c, bool gated);      // the form in which the tensor core applies e8m0 scales
cudaError_t launch_fp8_mx(const GemmCall& c, bool gated, const MxPlan& p, cudaStream_t s);
void plan_fp8_few(moe_linear* L);                       // sets few_*, from the weights' shape
bool few_tokens(const GemmCall& c);                     // whether the few-token form takes the call
cudaError_t launch_fp8_few(const GemmCall& c, bool gated, cudaStream_t s);

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();   // NULL when the driver has none

}  // namespace moe
