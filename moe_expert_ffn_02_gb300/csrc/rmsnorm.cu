// Residual addition, root-mean-square norm and 1x128 E4M3 quantisation in one
// pass over the data.
//
//   v = x + r              fp32, unrounded (r optional; v stored once rounded)
//   n = v * rsqrt(mean(v^2) + eps) * w
//   y = round(n)                                   (optional)
//   s = amax over 128 channels / 448, q = E4M3(n / s)    (optional)
//
// Bound by HBM: a row is read once (x and r), kept in registers across the
// row's sum of squares, and every output is written once: 7 bytes per element
// for bf16 streams with codes only.  One CTA per row; a lane holds 8
// consecutive channels, so 16 lanes hold one scale group and its amax takes
// four shuffles.  VPT vectors of 8 channels per thread keep 2 * VPT 16-byte
// loads in flight.
#include "dense_internal.cuh"

namespace moe {
namespace {

struct NormArgs {
    int cols;
    float eps, inv_cols;
    const void* x;
    const void* r;
    const float* w;
    void* ro;
    void* y;
    uint8_t* q;
    void* s;
    int64_t ldx, ldr, ldro, ldy, ldq, lds;
    bool e8m0;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_bits_to_f32(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// 8 channels c..c+7 of a row; VEC: 16-byte accesses (rows 16-byte aligned and
// all 8 channels inside), otherwise element by element with zeros past n.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&v)[8]) {
    if (vec) {
        if constexpr (sizeof(T) == 2) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
            const float4 a = reinterpret_cast<const float4*>(p)[0];
            const float4 b = reinterpret_cast<const float4*>(p)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32<T>(p[i]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool vec, const float (&v)[8]) {
    if (vec) {
        if constexpr (sizeof(T) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)from_f32<uint16_t>(v[2 * i]) | ((uint32_t)from_f32<uint16_t>(v[2 * i + 1]) << 16);
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
}

template <typename TX, typename TR, int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(NormArgs a, bool vec) {
    __shared__ float part[32];
    const int64_t row = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const TX* x = static_cast<const TX*>(a.x) + row * a.ldx;
    const TR* r = a.r ? static_cast<const TR*>(a.r) + row * a.ldr : nullptr;
    TR* ro = a.ro ? static_cast<TR*>(a.ro) + row * a.ldro : nullptr;
    float v[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * 8, n = a.cols - c;
        if (n > 0) load8<TX>(x + c, n, vec && n >= 8, v[i]);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
    if (r) {
        float u[VPT][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * 8, n = a.cols - c;
            if (n > 0) load8<TR>(r + c, n, vec && n >= 8, u[i]);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * 8, n = a.cols - c;
            if (n > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] += u[i][e];
                if (ro) store8<TR>(ro + c, n, vec && n >= 8, v[i]);
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    const int nw = blockDim.x >> 5;
    float tot = lane < nw ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xFFFFFFFFu, tot, o);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(tot, a.inv_cols, a.eps)));

    TX* y = a.y ? static_cast<TX*>(a.y) + row * a.ldy : nullptr;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * 8, n = a.cols - c;
        float w[8];
        if (n > 0) load8<float>(a.w + c, n, vec && n >= 8, w);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = n > e ? v[i][e] * rstd * w[e] : 0.f;
        if (y && n > 0) store8<TX>(y + c, n, vec && n >= 8, v[i]);
        if (a.q) {                                     // uniform: every lane takes part in the shuffles
            float am = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) am = max_nan(am, fabsf(v[i][e]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
            uint32_t held;
            const float sc = group_scale(am, a.e8m0, held);
            // n / s as n * (1 / s): within one ulp of the quotient, far inside the code spacing
            const float is = inv_scale(sc);
            if (n > 0) {
                const uint32_t lo = pack4_e4m3(v[i][0] * is, v[i][1] * is, v[i][2] * is, v[i][3] * is);
                const uint32_t hi = pack4_e4m3(v[i][4] * is, v[i][5] * is, v[i][6] * is, v[i][7] * is);
                uint8_t* q = a.q + row * a.ldq + c;
                if (n >= 8) {                          // code rows lie on 16-byte strides
                    *reinterpret_cast<uint2*>(q) = make_uint2(lo, hi);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < n) q[e] = (uint8_t)((e < 4 ? lo >> (8 * e) : hi >> (8 * (e - 4))) & 0xFFu);
                }
                if ((lane & 15) == 0) {
                    const int64_t at = (int64_t)(c / QB) * a.lds + row;
                    if (a.e8m0) static_cast<uint8_t*>(a.s)[at] = (uint8_t)held;
                    else static_cast<uint32_t*>(a.s)[at] = held;
                }
            }
        }
    }
}

template <typename TX, typename TR, int VPT>
cudaError_t go(const NormArgs& a, int rows, bool vec, cudaStream_t s) {
    const int vecs = (a.cols + 7) / 8;
    int threads = (vecs + VPT - 1) / VPT;
    threads = (threads + 31) / 32 * 32;
    return launch_pdl(rmsnorm_kernel<TX, TR, VPT>, dim3(rows), dim3(threads), 0, s, a, vec);
}

template <typename TX, typename TR>
cudaError_t pick(const NormArgs& a, int rows, bool vec, cudaStream_t s) {
    const int vecs = (a.cols + 7) / 8;
    if (vecs > 2048) return go<TX, TR, 4>(a, rows, vec, s);
    if (vecs > 1024) return go<TX, TR, 2>(a, rows, vec, s);
    return go<TX, TR, 1>(a, rows, vec, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const moe_rmsnorm_args* p, cudaStream_t s) {
    NormArgs a;
    a.cols = p->cols;
    a.eps = p->eps;
    a.inv_cols = 1.0f / (float)p->cols;
    a.x = p->x; a.r = p->res; a.w = p->weight; a.ro = p->res_out; a.y = p->y; a.q = p->out.q; a.s = p->out.s;
    a.ldx = p->ldx; a.ldr = p->ld_res; a.ldro = p->ld_res_out; a.ldy = p->ldy; a.ldq = p->out.ldq; a.lds = p->out.lds;
    a.e8m0 = p->out.scale_type == MOE_SCALE_E8M0;
    // 16-byte accesses need every row of every fp operand on a 16-byte boundary
    auto ok = [](const void* q, int64_t ld, int es) {
        return !q || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && (ld * es) % 16 == 0);
    };
    const int xs = p->x_type == MOE_F32 ? 4 : 2, rs = p->res_type == MOE_F32 ? 4 : 2;
    const bool vec = ok(a.x, a.ldx, xs) && ok(a.r, a.ldr, rs) && ok(a.ro, a.ldro, rs) && ok(a.y, a.ldy, xs) &&
                     ok(a.w, 0, 4);
    if (p->x_type == MOE_F32) return pick<float, float>(a, p->rows, vec, s);
    if (p->res_type == MOE_F32) return pick<uint16_t, float>(a, p->rows, vec, s);
    return pick<uint16_t, uint16_t>(a, p->rows, vec, s);
}

}  // namespace moe
