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
// Four forms.  Few rows: one CTA per row, as many threads as vectors (latency
// counts; a row of 7168 takes 2.5 us).  Many rows: persistent CTAs with a ring of
// rows in shared memory, filled by bulk copies that run ahead of the
// arithmetic; loading straight into registers leaves HBM idle while a CTA waits
// for its row's sum (8192 x 7168 bf16: 102 us, now 67 to 69, 0.91 of the copy
// bandwidth).  Rows off the 16-byte grid: contiguous two- and four-byte accesses,
// a warp per scale group, and the ring with each row's 16-byte window (8192 x 7001
// bf16 141 us, without residual 100, fp32 134; bound by its instructions and two-byte accesses).
// Short rows (256 channels at most): a warp per row.
#include "dense_internal.cuh"

#include <algorithm>
#include <atomic>

namespace moe {
namespace {

__device__ uint32_t g_status;                // MOE_DEV_WAIT_TIMEOUT once a wait gave up, per device
std::atomic<uint32_t> g_wait_limit{LANDING_LIMIT_US};
std::atomic<bool> g_plant{false};            // moe_rmsnorm_debug_timeout, for the next ring-form call

constexpr int MAX_ROWS = 16;                 // ring stages, at most
constexpr int RING_BYTES = 96 * 1024;        // per CTA; two CTAs share an SM

struct NormArgs {
    int rows, cols;
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

struct RingArgs {
    int stages;
    uint32_t xb, rb;           // bytes of a stage's x and r
    uint32_t wait_limit;
    bool plant;                // moe_rmsnorm_debug_timeout: the first CTA's second row never counts as copied
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

// 8 channels, 16-byte accesses.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
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
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
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
}

// n = v * rstd * w of one vector (8 channels from c), its outputs and, with 15 neighbouring lanes,
// its group's scale.  Every lane of the warp calls it; in: c lies inside the row.
template <typename TX>
__device__ __forceinline__ void finish8(const NormArgs& a, int64_t row, int c, bool in, float (&v)[8], const float (&w)[8],
                                        float rstd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = in ? v[e] * rstd * w[e] : 0.f;
    if (a.y && in) store8<TX>(static_cast<TX*>(a.y) + row * a.ldy + c, v);
    if (a.q) {
        float am = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) am = max_nan(am, fabsf(v[e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
        uint32_t held;
        // n / s as n * (1 / s): within one ulp of the quotient, far inside the code spacing
        const float is = inv_scale(group_scale(am, a.e8m0, held));
        if (in) {
            *reinterpret_cast<uint2*>(a.q + row * a.ldq + c) =        // code rows lie on 16-byte strides
                make_uint2(pack4_e4m3(v[0] * is, v[1] * is, v[2] * is, v[3] * is), pack4_e4m3(v[4] * is, v[5] * is, v[6] * is, v[7] * is));
            if ((threadIdx.x & 15) == 0) {
                const int64_t at = (int64_t)(c / QB) * a.lds + row;
                if (a.e8m0) static_cast<uint8_t*>(a.s)[at] = (uint8_t)held;
                else static_cast<uint32_t*>(a.s)[at] = held;
            }
        }
    }
}

// Sum of ss over the row's threads (a warp, or the CTA with one barrier) and 1 / sqrt(mean + eps).
template <bool WARP>
__device__ __forceinline__ float row_rstd(const NormArgs& a, float ss, float* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (!WARP) {
        if (lane == 0) part[warp] = ss;
        __syncthreads();
        ss = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    }
    return __fdiv_rn(1.0f, __fsqrt_rn(fmaf(ss, a.inv_cols, a.eps)));
}

// A row's place: one per CTA, or (WARP: short rows, many of them) one per warp.
struct RowOf {
    int64_t row;
    int tid, threads, warp, warps;
};
template <bool WARP>
__device__ __forceinline__ RowOf row_of() {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (WARP) return RowOf{(int64_t)blockIdx.x * (blockDim.x >> 5) + warp, lane, 32, 0, 1};
    return RowOf{blockIdx.x, (int)threadIdx.x, (int)blockDim.x, warp, (int)(blockDim.x >> 5)};
}

template <typename TX, typename TR, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rmsnorm_kernel(NormArgs a) {
    __shared__ float part[32];
    const RowOf at = row_of<WARP>();
    const int64_t row = at.row;
    pdl_trigger();
    pdl_wait();
    if (WARP && row >= a.rows) return;
    const TX* x = static_cast<const TX*>(a.x) + row * a.ldx;
    const TR* r = a.r ? static_cast<const TR*>(a.r) + row * a.ldr : nullptr;
    TR* ro = a.ro ? static_cast<TR*>(a.ro) + row * a.ldro : nullptr;
    float v[VPT][8] = {};
    auto channel = [&](int i) { return (i * at.threads + at.tid) * 8; };
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (channel(i) < a.cols) load8<TX>(x + channel(i), v[i]);
    if (r) {
        float u[VPT][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (channel(i) < a.cols) load8<TR>(r + channel(i), u[i]);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (channel(i) >= a.cols) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] += u[i][e];
            if (ro) store8<TR>(ro + channel(i), v[i]);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    const float rstd = row_rstd<WARP>(a, ss, part);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = channel(i);
        float w[8] = {};
        if (c < a.cols) load8<float>(a.w + c, w);
        finish8<TX>(a, row, c, c < a.cols, v[i], w, rstd);
    }
}

// Many rows.  Row i of this CTA lies in stage i % stages: x, then r.  Every thread has read its
// part of a stage before the barrier in row_rstd, so the stage is refilled right after it.  A thread
// that gave up waiting for a row stores nothing of it, and raises the row's flag before that barrier;
// after it all threads see the flag and leave.  Sums and flags have two buffers, because the next
// row's may come early (a flag raised at any time let threads of one row decide differently).

// The ring's barriers; the planted one expects an arrival more than it gets.
__device__ __forceinline__ void init_ring(uint64_t* full, const RingArgs& ra) {
    for (int s = 0; s < ra.stages; ++s) mbar_init(&full[s], ra.plant && blockIdx.x == 0 && s == 1 ? 2 : 1);
    fence_mbar_init();
}

// Thread 0, before a CTA that gave up at `row` in stage st leaves: the copies of that row and of those requested
// after it land.
__device__ __forceinline__ void land(uint64_t* full, const RingArgs& ra, int64_t row, int rows, int st, uint32_t phase) {
    if (ra.plant && blockIdx.x == 0) mbar_arrive(&full[1]);
    for (int s = 0; s < ra.stages && row < rows; ++s, row += gridDim.x) {
        mbar_wait_bounded(&full[st], phase, LANDING_LIMIT_US, &g_status, nullptr);
        if (++st == ra.stages) { st = 0; phase ^= 1u; }
    }
}

template <typename TX, typename TR, int VPT>
__global__ void __launch_bounds__(512, VPT > 2 ? 1 : 2) rmsnorm_stream_kernel(NormArgs a, RingArgs ra) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float part[2][32];
    __shared__ uint64_t full[MAX_ROWS];
    __shared__ volatile int abort_flag, gave_up[2];
    const int rows = a.rows, stages = ra.stages;
    const uint32_t xb = ra.xb, rb = ra.rb;
    if (threadIdx.x == 0) {
        abort_flag = gave_up[0] = gave_up[1] = 0;
        init_ring(full, ra);
    }
    pdl_trigger();
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
    float w[VPT][8];                           // the caller's memory, like the rows: read after the wait, under the first copies
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * 8;
        if (c < a.cols) load8<float>(a.w + c, w[i]);
    }
    int st = 0, par = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        float v[VPT][8];
        float ss = 0.f;
        if (mbar_wait_bounded(&full[st], phase, ra.wait_limit, &g_status, &abort_flag)) {
            const TX* x = reinterpret_cast<const TX*>(ring + (size_t)st * (xb + rb));
            const TR* r = reinterpret_cast<const TR*>(ring + (size_t)st * (xb + rb) + xb);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (i * blockDim.x + threadIdx.x) * 8;
                if (c < a.cols) {
                    load8<TX>(x + c, v[i]);
                    if (rb) {
                        float u[8];
                        load8<TR>(r + c, u);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[i][e] += u[e];
                        if (a.ro) store8<TR>(static_cast<TR*>(a.ro) + row * a.ldro + c, v[i]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
                }
            }
        } else {
            gave_up[par] = 1;
        }
        const float rstd = row_rstd<false>(a, ss, part[par]);
        if (gave_up[par]) {                    // seen by every thread, or by none
            if (threadIdx.x == 0) land(full, ra, row, rows, st, phase);
            break;
        }
        par ^= 1;
        const int64_t next = row + (int64_t)stages * gridDim.x;
        if (threadIdx.x == 0 && next < rows) fetch(next, st);
        if (++st == stages) { st = 0; phase ^= 1u; }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * 8;
            finish8<TX>(a, row, c, c < a.cols, v[i], w[i], rstd);
        }
    }
}

// Rows that do not lie on 16-byte boundaries (odd widths, views).  A warp takes whole scale groups, its
// lanes consecutive channels, so that the two- and four-byte accesses of a warp are contiguous: GPW groups
// of 4 x 32 channels per warp.
template <int GPW>
struct Narrow {
    static constexpr bool KEEP_W = GPW <= 4;               // this thread's weights in registers
    float v[GPW][4], w[KEEP_W ? GPW : 1][4];
    int warp, warps;
    __device__ __forceinline__ int channel(int i, int k) const { return (warp + i * warps) * QB + 32 * k + (threadIdx.x & 31); }

    __device__ __forceinline__ void load_weights(const NormArgs& a) {
        if constexpr (KEEP_W) {
#pragma unroll
            for (int i = 0; i < GPW; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) w[i][k] = channel(i, k) < a.cols ? a.w[channel(i, k)] : 0.f;
        }
    }

    // v = x + r, in place of r's row where ro is given; the sum of squares of this thread's part.
    template <typename TX, typename TR>
    __device__ __forceinline__ float take(const NormArgs& a, const TX* x, const TR* r, TR* ro) {
#pragma unroll
        for (int i = 0; i < GPW; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = channel(i, k) < a.cols ? to_f32<TX>(x[channel(i, k)]) : 0.f;
        if (r) {
            float u[GPW][4];
#pragma unroll
            for (int i = 0; i < GPW; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) u[i][k] = channel(i, k) < a.cols ? to_f32<TR>(r[channel(i, k)]) : 0.f;
#pragma unroll
            for (int i = 0; i < GPW; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[i][k] += u[i][k];
                    if (ro && channel(i, k) < a.cols) ro[channel(i, k)] = from_f32<TR>(v[i][k]);
                }
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < GPW; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) ss = fmaf(v[i][k], v[i][k], ss);
        return ss;
    }

    // The groups' chains (largest of 32 lanes, scale, codes) run side by side.
    template <typename TX>
    __device__ __forceinline__ void finish(const NormArgs& a, int64_t row, float rstd) {
        float am[GPW];
#pragma unroll
        for (int i = 0; i < GPW; ++i) {
            am[i] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = channel(i, k);
                if (c < a.cols) {
                    v[i][k] = v[i][k] * rstd * (KEEP_W ? w[KEEP_W ? i : 0][k] : a.w[c]);
                    if (a.y) static_cast<TX*>(a.y)[row * a.ldy + c] = from_f32<TX>(v[i][k]);
                }
                am[i] = max_nan(am[i], fabsf(v[i][k]));
            }
        }
        if (!a.q) return;                                  // uniform: every lane takes part in the shuffles
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < GPW; ++i) am[i] = max_nan(am[i], __shfl_xor_sync(0xFFFFFFFFu, am[i], o));
        uint32_t held[GPW], mine[GPW], out[GPW];
#pragma unroll
        for (int i = 0; i < GPW; ++i) {
            const float is = inv_scale(group_scale(am[i], a.e8m0, held[i]));
            mine[i] = pack4_e4m3(v[i][0] * is, v[i][1] * is, v[i][2] * is, v[i][3] * is);
            out[i] = 0;
        }
        // lane l holds channels l, 32 + l, ..; it stores channels 4 l .. 4 l + 3, four bytes at a time
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < GPW; ++i)
                out[i] |= ((__shfl_sync(0xFFFFFFFFu, mine[i], (4 * lane + j) & 31) >> (8 * (lane >> 3))) & 0xFFu) << (8 * j);
#pragma unroll
        for (int i = 0; i < GPW; ++i) {
            const int g = warp + i * warps, c = g * QB + 4 * lane;
            uint8_t* q = a.q + row * a.ldq + c;
            if (c + 4 <= a.cols) {
                *reinterpret_cast<uint32_t*>(q) = out[i];
            } else {
                for (int j = 0; c + j < a.cols; ++j) q[j] = (uint8_t)(out[i] >> (8 * j));
            }
            if (lane == 0 && g * QB < a.cols) {
                const int64_t at = (int64_t)g * a.lds + row;
                if (a.e8m0) static_cast<uint8_t*>(a.s)[at] = (uint8_t)held[i];
                else static_cast<uint32_t*>(a.s)[at] = held[i];
            }
        }
    }
};

template <typename TX, typename TR, int GPW, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rmsnorm_narrow_kernel(NormArgs a) {
    __shared__ float part[32];
    const RowOf at = row_of<WARP>();
    pdl_trigger();
    Narrow<GPW> n;
    n.warp = at.warp;
    n.warps = at.warps;
    pdl_wait();
    if (WARP && at.row >= a.rows) return;
    n.load_weights(a);
    const float ss = n.template take<TX, TR>(a, static_cast<const TX*>(a.x) + at.row * a.ldx,
                                             a.r ? static_cast<const TR*>(a.r) + at.row * a.ldr : nullptr,
                                             a.ro ? static_cast<TR*>(a.ro) + at.row * a.ldro : nullptr);
    n.template finish<TX>(a, at.row, row_rstd<WARP>(a, ss, part));
}

// Many long rows off the 16-byte grid: the ring form with each row's 16-byte window (the bytes around it
// up to the next boundaries, which belong to its neighbours).  A row whose window would leave the tensor,
// the first or the last, is copied by the threads instead.
struct Window {
    const uint8_t* from;
    uint32_t bytes, skip;                              // window, and the row's offset in it
    bool inside;
};
__device__ __forceinline__ Window window_of(const void* base, int64_t ld, int64_t row, int rows, int cols, int es) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base), hi = lo + (((int64_t)rows - 1) * ld + cols) * es;
    const uintptr_t at = lo + row * ld * es, from = at & ~uintptr_t(15), to = (at + (uintptr_t)cols * es + 15) & ~uintptr_t(15);
    return Window{reinterpret_cast<const uint8_t*>(from), (uint32_t)(to - from), (uint32_t)(at - from), from >= lo && to <= hi};
}

template <typename TX, typename TR, int GPW>
__global__ void __launch_bounds__(1024) rmsnorm_narrow_stream_kernel(NormArgs a, RingArgs ra) {
    extern __shared__ __align__(128) uint8_t ring[];       // [stage][xb | rb]: room for the largest windows
    __shared__ float part[2][32];
    __shared__ uint64_t full[MAX_ROWS];
    __shared__ volatile int abort_flag, gave_up[2];
    const int stages = ra.stages;
    const uint32_t xb = ra.xb, rb = ra.rb;
    if (threadIdx.x == 0) {
        abort_flag = gave_up[0] = gave_up[1] = 0;
        init_ring(full, ra);
    }
    pdl_trigger();
    Narrow<GPW> n;
    n.warp = threadIdx.x >> 5;
    n.warps = blockDim.x >> 5;
    __syncthreads();
    pdl_wait();
    auto x_window = [&](int64_t row) { return window_of(a.x, a.ldx, row, a.rows, a.cols, (int)sizeof(TX)); };
    auto r_window = [&](int64_t row) { return window_of(a.r, a.ldr, row, a.rows, a.cols, (int)sizeof(TR)); };
    auto fetch = [&](int64_t row, int st) {
        const Window x = x_window(row);
        const Window r = rb ? r_window(row) : Window{nullptr, 0, 0, false};
        uint8_t* at = ring + (size_t)st * (xb + rb);
        mbar_arrive_expect_tx(&full[st], (x.inside ? x.bytes : 0) + (r.inside ? r.bytes : 0));
        if (x.inside) bulk_g2s(at, x.from, x.bytes, &full[st]);
        if (r.inside) bulk_g2s(at + xb, r.from, r.bytes, &full[st]);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < stages && (int64_t)blockIdx.x + (int64_t)s * gridDim.x < a.rows; ++s)
            fetch((int64_t)blockIdx.x + (int64_t)s * gridDim.x, s);
    n.load_weights(a);
    int st = 0, par = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float ss = 0.f;
        if (mbar_wait_bounded(&full[st], phase, ra.wait_limit, &g_status, &abort_flag)) {
            uint8_t* at = ring + (size_t)st * (xb + rb);
            const Window xw = x_window(row), rw = rb ? r_window(row) : Window{nullptr, 0, 0, true};
            const TX* x = xw.inside ? reinterpret_cast<const TX*>(at + xw.skip) : static_cast<const TX*>(a.x) + row * a.ldx;
            const TR* r = !rb ? nullptr : rw.inside ? reinterpret_cast<const TR*>(at + xb + rw.skip)
                                                    : static_cast<const TR*>(a.r) + row * a.ldr;
            ss = n.template take<TX, TR>(a, x, r, a.ro ? static_cast<TR*>(a.ro) + row * a.ldro : nullptr);
        } else {
            gave_up[par] = 1;
        }
        const float rstd = row_rstd<false>(a, ss, part[par]);
        if (gave_up[par]) {
            if (threadIdx.x == 0) land(full, ra, row, a.rows, st, phase);
            break;
        }
        par ^= 1;
        const int64_t next = row + (int64_t)stages * gridDim.x;
        if (threadIdx.x == 0 && next < a.rows) fetch(next, st);
        if (++st == stages) { st = 0; phase ^= 1u; }
        n.template finish<TX>(a, row, rstd);
    }
}

int sm_count(cudaError_t& e) {
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <typename TX, typename TR, int VPT>
cudaError_t go(const NormArgs& a, cudaStream_t s) {
    const int vecs = a.cols / 8, threads = ((vecs + VPT - 1) / VPT + 31) / 32 * 32;
    return launch_pdl(rmsnorm_kernel<TX, TR, VPT, false>, dim3(a.rows), dim3(threads), 0, s, a);
}

RingArgs ring_args(int stages, uint32_t xb, uint32_t rb) {
    const bool plant = g_plant.load(std::memory_order_relaxed) && g_plant.exchange(false);
    return RingArgs{stages, xb, rb, g_wait_limit.load(std::memory_order_relaxed), plant};
}

template <typename TX, typename TR, int GPW>
cudaError_t go_narrow(const NormArgs& a, bool warp, int stages, uint32_t xb, uint32_t rb, int ctas, cudaStream_t s) {
    if constexpr (GPW <= 2)
        if (warp) return launch_pdl(rmsnorm_narrow_kernel<TX, TR, GPW, true>, dim3((a.rows - 1) / 8 + 1), dim3(256), 0, s, a);
    const int groups = (a.cols + QB - 1) / QB;
    const dim3 threads((groups + GPW - 1) / GPW * 32);
    if constexpr (GPW > 1)
        if (stages) {
            cudaError_t e = ensure_smem_limit<rmsnorm_narrow_stream_kernel<TX, TR, GPW>>(RING_BYTES);
            if (e != cudaSuccess) return e;
            return launch_pdl(rmsnorm_narrow_stream_kernel<TX, TR, GPW>, dim3(ctas), threads, (size_t)stages * (xb + rb), s, a,
                              ring_args(stages, xb, rb));
        }
    return launch_pdl(rmsnorm_narrow_kernel<TX, TR, GPW, false>, dim3(a.rows), threads, 0, s, a);
}

template <typename TX, typename TR, int VPT>
cudaError_t go_stream(const NormArgs& a, int threads, int stages, uint32_t xb, uint32_t rb, int ctas, cudaStream_t s) {
    cudaError_t e = ensure_smem_limit<rmsnorm_stream_kernel<TX, TR, VPT>>(RING_BYTES);
    if (e != cudaSuccess) return e;
    return launch_pdl(rmsnorm_stream_kernel<TX, TR, VPT>, dim3(ctas), dim3(threads), (size_t)stages * (xb + rb), s, a,
                      ring_args(stages, xb, rb));
}

// vec: every row on 16-byte boundaries and a whole number of 16-byte vectors.
template <typename TX, typename TR>
cudaError_t pick(const NormArgs& a, bool vec, cudaStream_t s) {
    cudaError_t e;
    const int sms = sm_count(e);
    if (e != cudaSuccess) return e;
    // rows of up to 256 channels: a warp each, once there are enough of them to give every SM some (8192 x
    // 128: 3.7 us, one CTA per row 9.2; 2000 x 500: 5.6 against 3.9)
    const bool warp = a.cols <= 256 && a.rows >= 2 * sms;
    // rings: room for a row's window, and at least two rows of every CTA
    uint32_t xb = (uint32_t)a.cols * sizeof(TX), rb = a.r ? (uint32_t)a.cols * sizeof(TR) : 0u;
    if (!vec) {
        xb = (xb + 15) / 16 * 16 + 16;
        rb = rb ? (rb + 15) / 16 * 16 + 16 : 0u;
    }
    if (vec) {
        const int vecs = a.cols / 8, vpt = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
        if (!warp && vecs <= 2048) {
            const int threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
            // CTAs per SM: two of 512 threads; more where rows are short, up to 1024 threads and 192 KB of rings
            const int per_sm = std::max(vpt == 4 ? 1 : 2, std::min(8, 1024 / threads));
            const int stages = std::min(MAX_ROWS, (int)(std::min(RING_BYTES, 2 * RING_BYTES / per_sm) / (xb + rb)));
            const int ctas = per_sm * sms;
            if (stages >= 2 && a.rows >= 2 * ctas) {
                if (vpt == 1) return go_stream<TX, TR, 1>(a, threads, stages, xb, rb, ctas, s);
                if (vpt == 2) return go_stream<TX, TR, 2>(a, threads, stages, xb, rb, ctas, s);
                return go_stream<TX, TR, 4>(a, threads, stages, xb, rb, ctas, s);
            }
        }
        if (vecs > 2048) return go<TX, TR, 4>(a, s);
        if (vecs > 1024) return go<TX, TR, 2>(a, s);
        if (warp) return launch_pdl(rmsnorm_kernel<TX, TR, 1, true>, dim3((a.rows - 1) / 8 + 1), dim3(256), 0, s, a);
        return go<TX, TR, 1>(a, s);
    }
    const int groups = (a.cols + QB - 1) / QB;
    const int gpw = warp ? groups : groups <= 8 ? 1 : groups <= 16 ? 2 : groups <= 128 ? 4 : 8;
    int stages = 0, ctas = 0;
    if (!warp && gpw > 1) {
        const int threads = (groups + gpw - 1) / gpw * 32, per_sm = std::max(1, std::min(8, 1024 / threads));
        stages = std::min(MAX_ROWS, (int)(std::min(RING_BYTES, 2 * RING_BYTES / per_sm) / (xb + rb)));
        ctas = per_sm * sms;
        if (stages < 2 || a.rows < 2 * ctas) stages = 0;
    }
    if (gpw == 1) return go_narrow<TX, TR, 1>(a, warp, stages, xb, rb, ctas, s);
    if (gpw == 2) return go_narrow<TX, TR, 2>(a, warp, stages, xb, rb, ctas, s);
    if (gpw <= 4) return go_narrow<TX, TR, 4>(a, warp, stages, xb, rb, ctas, s);
    return go_narrow<TX, TR, 8>(a, warp, stages, xb, rb, ctas, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const moe_rmsnorm_args* p, cudaStream_t s) {
    NormArgs a;
    a.rows = p->rows;
    a.cols = p->cols;
    a.eps = p->eps;
    a.inv_cols = 1.0f / (float)p->cols;
    a.x = p->x; a.r = p->res; a.w = p->weight; a.ro = p->res_out; a.y = p->y; a.q = p->out.q; a.s = p->out.s;
    a.ldx = p->ldx; a.ldr = p->ld_res; a.ldro = p->ld_res_out; a.ldy = p->ldy; a.ldq = p->out.ldq; a.lds = p->out.lds;
    a.e8m0 = p->out.scale_type == MOE_SCALE_E8M0;
    // 16-byte accesses need every row of every floating operand on a 16-byte boundary
    auto ok = [](const void* q, int64_t ld, int es) {
        return !q || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && (ld * es) % 16 == 0);
    };
    const int xs = p->x_type == MOE_F32 ? 4 : 2, rs = p->res_type == MOE_F32 ? 4 : 2;
    const bool vec = a.cols % 8 == 0 && ok(a.x, a.ldx, xs) && ok(a.r, a.ldr, rs) && ok(a.ro, a.ldro, rs) && ok(a.y, a.ldy, xs) &&
                     ok(a.w, 0, 4);
    if (p->x_type == MOE_F32) return pick<float, float>(a, vec, s);
    if (p->res_type == MOE_F32) return pick<uint16_t, float>(a, vec, s);
    return pick<uint16_t, uint16_t>(a, vec, s);
}

void norm_set_wait_limit(uint32_t us) { g_wait_limit.store(us, std::memory_order_relaxed); }
void norm_plant_timeout() { g_plant.store(true); }
cudaError_t norm_status_word(uint32_t** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_status); }

}  // namespace moe
