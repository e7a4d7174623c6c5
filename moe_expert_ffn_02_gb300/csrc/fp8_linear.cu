// Plain FP8 projection: choice of the tile width, and the weights' image.
#include <mutex>

#include "fp8_gemm.cuh"

namespace moe {
namespace dg {

// Weight rows per tile, and K ranges: few token tiles take narrow tiles, so that every SM streams a
// share of the weights, or split K where rows are few and long; many take wide ones, which reuse the
// tokens.  A tile's K block takes the draining of its columns, or its copies.
static Plan plan_plain(const GemmCall& c, const Args& a) {
    const int sms = c.lin->num_sms, rows = c.lin->rows;
    const int mt = (c.M + BM - 1) / BM;
    Plan best = {};
    double best_us = 0;
    for (int bn = 16; bn <= BUF_COLS; bn += 16) {
        const int grp = bn <= 32 ? 8 : bn <= 64 ? 4 : bn <= 128 ? 2 : 1;
        if (grp == 1 && bn != 256) continue;                   // 256: both halves in whole scale blocks
        if (2 * stage_cost(grp, bn, a.a_rows) > ring_max()) continue;
        const int nt = (rows + bn - 1) / bn, groups = (a.kt + grp - 1) / grp;
        const long long units = (long long)mt * nt;
        if (units > 0x3FFFFFFF) continue;
        const double drain = grp == 1 ? 0.42 : grp == 2 ? 0.246 : 0.15;
        for (int S = 1; S <= 8 && S <= groups; S *= 2) {
            if (S > 1 && ((bn != 128 && bn != 256) || units > cluster_slots(sms, S))) break;
            const double kr = std::min<double>(a.kt, (double)grp * ((groups + S - 1) / S));
            const double us = plan_us(S > 1 ? 1.0 : (double)((units + sms - 1) / sms), kr, std::max(drain, copy_us(bn, a.a_rows)),
                                      0.965, memory_bytes(c, false)) +
                              join_us(false, bn, S, c.M, (double)units * S);
            if (best.bn == 0 || us < best_us) {
                best_us = us;
                best = Plan{grp, bn, S, (int)units, nt, S, us};
            }
        }
    }
    return best;
}

}  // namespace dg

cudaError_t launch_fp8_linear(const GemmCall& c, cudaStream_t s) {
    using namespace dg;
    if (few_tokens(c)) return launch_fp8_few(c, false, s);
    Args a = base_args(c);
    const Plan p = plan_plain(c, a);
    if (!p.bn) return cudaErrorInvalidValue;
    const MxPlan mx = plan_fp8_mx(c, false);
    if (mx.bn && mx.us <= p.us) return launch_fp8_mx(c, false, mx, s);
    switch (p.grp) {
        case 1: return launch<1, false>(c, p, a, s);
        case 2: return launch<2, false>(c, p, a, s);
        case 4: return launch<4, false>(c, p, a, s);
        default: return launch<8, false>(c, p, a, s);
    }
}

// ------------------------------------------------------------------ weights' image
// [kt][rows_pad][128 B]: row r of K block kb at 128 (kb rows_pad + r), its
// 16-byte chunk c at position c ^ (r mod 8): the K-major, 128-byte-swizzled
// operand layout, so any 8-aligned run of rows of a K block is one contiguous
// bulk copy.  Gated: rows 16 j .. 16 j + 7 are gate features 8 j .. 8 j + 7, the next
// eight the same features' up rows, so one thread of the GEMM's epilogue holds both.
__global__ void linear_image_kernel(const uint8_t* __restrict__ w, const uint8_t* __restrict__ wu, int N, int K, int kt,
                                    int rows_pad, uint8_t* __restrict__ img) {
    const size_t n = (size_t)kt * rows_pad * 8;
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
        const int pos = (int)(i & 7);
        const size_t line = i >> 3;
        const int r = (int)(line % rows_pad), kb = (int)(line / rows_pad);
        const int k0 = kb * QB + (pos ^ (r & 7)) * 16;
        const int f = wu ? (r >> 4) * 8 + (r & 7) : r;
        const uint8_t* src = (wu && (r & 8)) ? wu : w;
        uint32_t v[4] = {0, 0, 0, 0};
        if (f < N && k0 < K) {
            const uint8_t* p = src + (size_t)f * K + k0;
            if (k0 + 16 <= K && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
                const uint4 u = *reinterpret_cast<const uint4*>(p);
                v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
            } else {
                for (int b = 0; b < 16; ++b)
                    if (k0 + b < K) v[b >> 2] |= (uint32_t)p[b] << (8 * (b & 3));
            }
        }
        reinterpret_cast<uint4*>(img)[i] = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

__global__ void linear_scales_kernel(const void* s, const void* su, int n, bool e8m0, float* __restrict__ out) {
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < (su ? 2 * n : n); i += gridDim.x * blockDim.x) {
        const void* src = i < n ? s : su;
        const int j = i < n ? i : i - n;
        out[i] = e8m0 ? e8m0_to_f32(static_cast<const uint8_t*>(src)[j]) : static_cast<const float*>(src)[j];
    }
}

// Scale-factor blocks for the tensor core's own scaling: 128 image rows x 4 K blocks in 512 bytes,
// row r at (r mod 32) * 16 + (r / 32) * 4, one byte per K block.
__global__ void linear_sf_kernel(const uint8_t* __restrict__ s, const uint8_t* __restrict__ su, int N, int kt, int rows_pad,
                                 uint8_t* __restrict__ out) {
    const int nrb = (rows_pad + QB - 1) / QB;
    const size_t n = (size_t)((kt + 3) / 4) * nrb * 512;
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
        const int b = (int)(i & 511), rb = (int)((i >> 9) % nrb), q = (int)((i >> 9) / nrb);
        const int r = rb * QB + ((b >> 2) & 3) * 32 + (b >> 4), kb = 4 * q + (b & 3);
        const int f = su ? (r >> 4) * 8 + (r & 7) : r;
        const uint8_t* src = su && (r & 8) ? su : s;
        out[i] = f < N && kb < kt ? src[(size_t)(f / QB) * kt + kb] : 127;
    }
}

cudaError_t launch_linear_repack(const moe_linear* L, const uint8_t* w, const void* s, const uint8_t* wu,
                                 const void* su, cudaStream_t st) {
    linear_image_kernel<<<8 * L->num_sms, 256, 0, st>>>(w, wu, L->d.out_features, L->d.in_features, L->kt, L->rows_pad,
                                                        L->w);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int n = (L->d.out_features + QB - 1) / QB * L->kt;
    linear_scales_kernel<<<L->num_sms, 256, 0, st>>>(s, su, n, L->d.scale_type == MOE_SCALE_E8M0, L->sw);
    e = cudaGetLastError();
    if (e != cudaSuccess || !L->wsf) return e;
    linear_sf_kernel<<<4 * L->num_sms, 256, 0, st>>>(static_cast<const uint8_t*>(s), static_cast<const uint8_t*>(su),
                                                     L->d.out_features, L->kt, L->rows_pad, L->wsf);
    return cudaGetLastError();
}

EncodeTiledFn tensor_map_encoder() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

}  // namespace moe
