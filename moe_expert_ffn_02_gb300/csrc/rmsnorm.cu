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
// for bf16 streams with codes only.  A lane holds 8 consecutive channels per
// vector, so 16 lanes hold one scale group and its amax takes four shuffles.
//
// Two forms.  Few rows: one CTA per row, as many threads as vectors (latency
// counts; a row of 7168 takes 2.7 us).  Many rows: persistent CTAs with a ring of
// rows in shared memory, filled by bulk copies that run ahead of the
// arithmetic; loading straight into registers leaves HBM idle while a CTA waits
// for its row's sum (8192 x 7168 bf16: 102 us).
#include "dense_internal.cuh"

#include <algorithm>

namespace moe {
namespace {

__device__ uint32_t g_status;                // MOE_DEV_WAIT_TIMEOUT once a wait gave up, per device
constexpr uint32_t WAIT_LIMIT_US = 2000000;

constexpr int MAX_ROWS = 16;                 // ring stages, at most
constexpr int RING_BYTES = 96 * 1024;        // per CTA; two CTAs share an SM

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

// n = v * rstd * w of one vector (8 channels from c), its outputs and, with 15 neighbouring lanes,
// its group's scale.  Every lane of the warp calls it: n <= 0 past the row's end.
template <typename TX>
__device__ __forceinline__ void finish8(const NormArgs& a, int64_t row, int c, int n, bool vec, float (&v)[8], const float (&w)[8],
                                        float rstd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = n > e ? v[e] * rstd * w[e] : 0.f;
    if (a.y && n > 0) store8<TX>(static_cast<TX*>(a.y) + row * a.ldy + c, n, vec && n >= 8, v);
    if (a.q) {
        float am = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) am = max_nan(am, fabsf(v[e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
        uint32_t held;
        // n / s as n * (1 / s): within one ulp of the quotient, far inside the code spacing
        const float is = inv_scale(group_scale(am, a.e8m0, held));
        if (n > 0) {
            const uint32_t lo = pack4_e4m3(v[0] * is, v[1] * is, v[2] * is, v[3] * is);
            const uint32_t hi = pack4_e4m3(v[4] * is, v[5] * is, v[6] * is, v[7] * is);
            uint8_t* q = a.q + row * a.ldq + c;
            if (n >= 8) {                              // code rows lie on 16-byte strides
                *reinterpret_cast<uint2*>(q) = make_uint2(lo, hi);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) q[e] = (uint8_t)((e < 4 ? lo >> (8 * e) : hi >> (8 * (e - 4))) & 0xFFu);
            }
            if ((threadIdx.x & 15) == 0) {
                const int64_t at = (int64_t)(c / QB) * a.lds + row;
                if (a.e8m0) static_cast<uint8_t*>(a.s)[at] = (uint8_t)held;
                else static_cast<uint32_t*>(a.s)[at] = held;
            }
        }
    }
}

// Sum of ss over the CTA's threads and 1 / sqrt(mean + eps); one CTA barrier.
__device__ __forceinline__ float row_rstd(const NormArgs& a, float ss, float* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    float tot = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xFFFFFFFFu, tot, o);
    return __fdiv_rn(1.0f, __fsqrt_rn(fmaf(tot, a.inv_cols, a.eps)));
}

template <typename TX, typename TR, int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(NormArgs a, bool vec) {
    __shared__ float part[32];
    const int64_t row = blockIdx.x;
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
    const float rstd = row_rstd(a, ss, part);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * 8, n = a.cols - c;
        float w[8];
        if (n > 0) load8<float>(a.w + c, n, vec && n >= 8, w);
        finish8<TX>(a, row, c, n, vec, v[i], w, rstd);
    }
}

// Many rows.  Row i of this CTA lies in stage i % stages: x, then r.  Every thread has read its
// part of a stage before the barrier in row_rstd, so the stage is refilled right after it.
template <typename TX, typename TR, int VPT>
__global__ void __launch_bounds__(512, VPT > 2 ? 1 : 2) rmsnorm_stream_kernel(NormArgs a, int rows, int stages, uint32_t xb, uint32_t rb) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float part[2][32];
    __shared__ uint64_t full[MAX_ROWS];
    __shared__ volatile int abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    pdl_trigger();
    float w[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * 8;
        if (c < a.cols) load8<float>(a.w + c, 8, true, w[i]);
    }
    __syncthreads();
    pdl_wait();
    auto fetch = [&](int64_t row, int st) {
        mbar_arrive_expect_tx(&full[st], xb + rb);
        bulk_g2s(ring + (size_t)st * (xb + rb), static_cast<const TX*>(a.x) + row * a.ldx, xb, &full[st]);
        if (rb) bulk_g2s(ring + (size_t)st * (xb + rb) + xb, static_cast<const TR*>(a.r) + row * a.ldr, rb, &full[st]);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < stages && (int64_t)blockIdx.x + (int64_t)s * gridDim.x < rows; ++s)
            fetch((int64_t)blockIdx.x + (int64_t)s * gridDim.x, s);
    int st = 0, par = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        // a wait that runs out raises the flag; the row's garbage is dropped after the barrier below
        mbar_wait_bounded(&full[st], phase, WAIT_LIMIT_US, &g_status, &abort_flag);
        const TX* x = reinterpret_cast<const TX*>(ring + (size_t)st * (xb + rb));
        const TR* r = reinterpret_cast<const TR*>(ring + (size_t)st * (xb + rb) + xb);
        float v[VPT][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * 8;
            if (c < a.cols) {
                load8<TX>(x + c, 8, true, v[i]);
                if (rb) {
                    float u[8];
                    load8<TR>(r + c, 8, true, u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] += u[e];
                    if (a.ro) store8<TR>(static_cast<TR*>(a.ro) + row * a.ldro + c, 8, true, v[i]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
            }
        }
        const float rstd = row_rstd(a, ss, part[par]);     // two buffers: the next row's sums may come early
        if (abort_flag) break;
        par ^= 1;
        const int64_t next = row + (int64_t)stages * gridDim.x;
        if (threadIdx.x == 0 && next < rows) fetch(next, st);
        if (++st == stages) { st = 0; phase ^= 1u; }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * 8;
            finish8<TX>(a, row, c, a.cols - c, true, v[i], w[i], rstd);
        }
    }
    if (abort_flag && threadIdx.x == 0)                    // copies in flight land before the CTA leaves
        for (int s = 0; s < stages; ++s) {
            mbar_wait_bounded(&full[st], phase, WAIT_LIMIT_US, &g_status, nullptr);
            if (++st == stages) { st = 0; phase ^= 1u; }
        }
}

template <typename TX, typename TR, int VPT>
cudaError_t go(const NormArgs& a, int rows, bool vec, cudaStream_t s) {
    const int vecs = (a.cols + 7) / 8;
    int threads = (vecs + VPT - 1) / VPT;
    threads = (threads + 31) / 32 * 32;
    return launch_pdl(rmsnorm_kernel<TX, TR, VPT>, dim3(rows), dim3(threads), 0, s, a, vec);
}

template <typename TX, typename TR, int VPT>
cudaError_t go_stream(const NormArgs& a, int rows, int threads, int stages, uint32_t xb, uint32_t rb, int ctas, cudaStream_t s) {
    cudaError_t e = ensure_smem_limit<rmsnorm_stream_kernel<TX, TR, VPT>>(RING_BYTES);
    if (e != cudaSuccess) return e;
    return launch_pdl(rmsnorm_stream_kernel<TX, TR, VPT>, dim3(ctas), dim3(threads), (size_t)stages * (xb + rb), s, a, rows, stages, xb, rb);
}

template <typename TX, typename TR>
cudaError_t pick(const NormArgs& a, int rows, bool vec, cudaStream_t s) {
    const int vecs = (a.cols + 7) / 8;
    // The ring form: rows of whole 16-byte vectors, enough of them for every CTA to have several, and
    // at least two in its ring.
    const uint32_t xb = (uint32_t)a.cols * sizeof(TX), rb = a.r ? (uint32_t)a.cols * sizeof(TR) : 0u;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int vpt = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
    if (vec && a.cols % 8 == 0 && vecs <= 2048 && 2 * (xb + rb) <= (uint32_t)RING_BYTES && rows >= 8 * sms) {
        const int threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
        // CTAs per SM: two of 512 threads; more where rows are short, up to 1024 threads and 192 KB of rings
        const int per_sm = std::max(vpt == 4 ? 1 : 2, std::min(8, 1024 / threads));
        const int ring = std::min(RING_BYTES, 2 * RING_BYTES / per_sm);
        const int stages = std::min(MAX_ROWS, (int)(ring / (xb + rb)));
        if (stages >= 2) {
            const int ctas = std::min(rows, per_sm * sms);
            if (vpt == 1) return go_stream<TX, TR, 1>(a, rows, threads, stages, xb, rb, ctas, s);
            if (vpt == 2) return go_stream<TX, TR, 2>(a, rows, threads, stages, xb, rb, ctas, s);
            return go_stream<TX, TR, 4>(a, rows, threads, stages, xb, rb, ctas, s);
        }
    }
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

cudaError_t norm_status_word(uint32_t** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_status); }

}  // namespace moe
