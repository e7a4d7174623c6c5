// Dense FP8 GEMM on the 5th-generation tensor cores (tcgen05, sm_103a),
// shared by the plain and the gated projection.
//
//   y[m][n] = sum over K blocks kb of  sa[kb][m] * sw[n / 128][kb] *
//             sum over the block's 128 channels of  A[m][k] * W[n][k]
//
// The inner sums are kind::f8f6f4 MMAs (E4M3 x E4M3, fp32 accumulate in tensor
// memory); each block's partial is scaled once, in fp32 registers, so nothing
// is rounded below 32 bits before the output.
//
// Operand roles: 128 tokens are the MMA's M (TMEM lanes), BN weight rows its N
// (TMEM columns), at every batch size.  A lane is one token, so sa is a
// per-thread scalar and sw is uniform per 16 columns.  BN is a multiple of 16
// chosen per call: it sets how many CTAs share the weights.  With few tokens
// every SM streams its own BN-row slice of W over the whole K, with no split
// sum to join; with many, BN = 256.
//
// A TMEM buffer holds 256 columns: GRP = 1, 2, 4 or 8 K blocks of up to
// 256 / GRP columns.  One commit covers the group, because a commit costs
// about 512 cycles of MMA time however little work it closes: narrow tiles need
// several blocks per commit.  Epilogue warp (quarter, half) owns 32 lanes and the
// half's columns of every block of the group, so blocks are added in K order
// into the same accumulators in every configuration and a row's result does
// not depend on BN or on the batch size.
//
// Warps: 0 copies (TMA for A, bulk copies for the pre-swizzled weight image), 1
// issues the MMAs, 2-3 idle, 4-11 drain.  Token tiles with fewer than 128 rows
// copy only those rows (rounded up to 8); the MMA reads whatever lies behind
// them in shared memory into TMEM lanes nobody reads.
#pragma once
#include "dense_internal.cuh"
#include "tcgen05.cuh"

#include <algorithm>

namespace moe {
namespace dg {

constexpr int BM = 128;
constexpr int CTRL_WARPS = 4, EPI_WARPS = 8;
constexpr int NTHREADS = (CTRL_WARPS + EPI_WARPS) * 32;
// setmaxnreg: launched at 168 per thread (384 x 168 = 64,512); control warps
// drop to 40, the drain warps rise to 232: 4*32*40 + 8*32*232 = 64,512
constexpr int CTRL_REGS = 40, EPI_REGS = 232;
static_assert(CTRL_WARPS * 32 * CTRL_REGS + EPI_WARPS * 32 * EPI_REGS <= NTHREADS * 168, "register split");
constexpr int BUF_COLS = 256;                 // TMEM columns of one buffer, two buffers
constexpr int MAX_STAGES = 8;
constexpr int STG_STRIDE = 20;                // floats between rows of a warp's 32 x 16 staging tile
constexpr int STG_BYTES = EPI_WARPS * 32 * STG_STRIDE * 4;
constexpr int MAX_CLUSTER = 8;
constexpr int AMAX_BYTES = 2 * MAX_CLUSTER * BM * 4;   // [unit parity][CTA rank][row]
constexpr int SMEM_MAX = 232448 - 2048;       // dynamic limit, minus static barriers
constexpr int RING_MAX = SMEM_MAX - 1024 - STG_BYTES - AMAX_BYTES - 2 * BM * 4;

struct Args {
    const uint8_t* w;         // weight image [kt][rows_pad][128]
    const float* sw;          // [1 or 2][nblk][kt]
    const void* sa;           // [kt][ld_sa] fp32 or e8m0
    int64_t ld_sa;
    int M, N, kt;             // N: output features
    int rows_pad, nblk;       // image rows; 128-row scale blocks per matrix
    int bn;                   // weight rows per tile
    int a_rows;               // token rows a tile copies (multiple of 8, at most 128)
    int stages;
    int n_nt;                 // weight tiles per token tile
    int n_units;
    bool e8m0;
    // plain
    void* y;
    int64_t ldy;
    bool y_f32, y_vec;
    // gated
    uint8_t* hq;
    int64_t ld_hq;
    void* hs;
    int64_t ld_hs;
    uint32_t* status;
    uint32_t wait_limit;
};

__device__ __forceinline__ uint32_t idesc_for(int n) {   // D f32, A = B = E4M3, K-major, M = 128
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// One fp32 value into a CTA of the cluster, counted on that CTA's mbarrier.
__device__ __forceinline__ void st_async_f32(uint32_t remote, float v, uint32_t remote_bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(remote),
                 "r"(__float_as_uint(v)), "r"(remote_bar)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint32_t limit_us, uint32_t* status,
                                                  volatile int* abort) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if (*abort) return false;
        if (global_ns() - t0 > (uint64_t)limit_us * 1000ull) {
            atomicOr(status, MOE_DEV_WAIT_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
}

__device__ __forceinline__ float load_sa(const Args& a, int kb, int row) {
    const int64_t at = (int64_t)kb * a.ld_sa + row;
    return a.e8m0 ? e8m0_to_f32(static_cast<const uint8_t*>(a.sa)[at]) : static_cast<const float*>(a.sa)[at];
}

// GRP: K blocks per TMEM buffer (and per commit).  A thread's pieces are 16
// columns each, 8 per buffer: PPK = 8 / GRP pieces per block.
template <int GRP, bool GATED>
__global__ void __launch_bounds__(NTHREADS, 1) fp8_gemm_kernel(const __grid_constant__ CUtensorMap ta, Args a) {
    constexpr int COLS = BUF_COLS / GRP;      // columns reserved per K block
    constexpr int HALF = COLS / 2;            // accumulators per thread
    constexpr int PPK = HALF / 16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int w_bytes = a.bn * 128, a_bytes = a.a_rows * 128;
    const int stage_bytes = GRP * (w_bytes + a_bytes);
    // behind the ring, in this order, so that the last block's 128-row operand read stays inside
    uint8_t* after = ring + a.stages * stage_bytes;
    float* stg_all = reinterpret_cast<float*>(after);
    float* amax_cta = reinterpret_cast<float*>(after + STG_BYTES);              // [half][128]
    float* amax_all = amax_cta + 2 * BM;                                        // [parity][rank][128]
    __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[2], tempty[2], xbar[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = GATED ? cluster_rank() : 0u, csize = GATED ? cluster_size() : 1u;
    const int first = blockIdx.x / csize, step = gridDim.x / csize;   // units go to clusters
    const int n_grp = (a.kt + GRP - 1) / GRP;

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], EPI_WARPS); mbar_init(&xbar[b], 1); }
        fence_mbar_init();
        abort_flag = 0;
    }
    if (warp == 1) tc::tmem_alloc(&tmem_slot, 512);
    tc::tc_fence_before();
    __syncthreads();
    if (GATED && csize > 1) cluster_sync();     // peers' barriers exist before anything is sent to them
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    volatile int* abort = &abort_flag;

    // unit -> token tile and first weight row
    auto unit_rows = [&](int u, int& m0, int& n0) {
        const int mt = u / a.n_nt;
        m0 = mt * BM;
        n0 = ((u - mt * a.n_nt) * (int)csize + (int)rank) * a.bn;
    };

    if (warp < CTRL_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTRL_REGS));
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ producer
            auto copy_w = [&](int stage, int n0, int g) {
                const int nk = min(GRP, a.kt - g * GRP);
                const int rows = max(0, min(a.bn, a.rows_pad - n0));
                mbar_arrive_expect_tx(&full[stage], (uint32_t)(nk * (rows * 128 + a_bytes)));
                if (rows > 0)
                    for (int i = 0; i < nk; ++i)
                        bulk_g2s(ring + stage * stage_bytes + i * w_bytes,
                                 a.w + ((size_t)(g * GRP + i) * a.rows_pad + n0) * 128, (uint32_t)(rows * 128),
                                 &full[stage]);
            };
            auto copy_a = [&](int stage, int m0, int g) {
                const int nk = min(GRP, a.kt - g * GRP);
                for (int i = 0; i < nk; ++i)
                    tma_load_2d(ring + stage * stage_bytes + GRP * w_bytes + i * a_bytes, &ta, (g * GRP + i) * QB, m0,
                                &full[stage]);
            };
            int stage = 0;
            uint32_t phase = 0, armed = 0, armed_par = 0;
            bool ok = true;
            // the weights do not depend on the preceding kernel: the first unit's stages are
            // requested before the wait for it
            int pre = 0;
            if (first < a.n_units) {
                int m0, n0;
                unit_rows(first, m0, n0);
                for (; pre < min(a.stages, n_grp); ++pre) copy_w(pre, n0, pre);
            }
            pdl_wait();
            for (int u = first; u < a.n_units && ok; u += step) {
                int m0, n0;
                unit_rows(u, m0, n0);
                for (int g = 0; g < n_grp; ++g) {
                    if (pre > 0) {
                        --pre;
                    } else {
                        if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, a.wait_limit, a.status, abort)) {
                            ok = false;
                            break;
                        }
                        copy_w(stage, n0, g);
                    }
                    copy_a(stage, m0, g);
                    armed |= 1u << stage;
                    armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == a.stages) { stage = 0; phase ^= 1u; }
                }
            }
            // every issued copy lands before the CTA exits
            for (int s = 0; s < a.stages; ++s)
                if ((armed >> s) & 1u) mbar_wait_bounded(&full[s], (armed_par >> s) & 1u, a.wait_limit, a.status, nullptr);
        } else if (warp == 1 && lane == 0) {
            // ------------------------------------------------ MMA issuer
            int stage = 0, buf = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true;
            const uint32_t idesc = idesc_for(a.bn);
            const uint64_t d0 = tc::sw128_desc(smem_addr(ring));
            for (int u = first; u < a.n_units && ok; u += step) {
                for (int g = 0; g < n_grp; ++g) {
                    if (!mbar_wait_bounded(&full[stage], phase, a.wait_limit, a.status, abort) ||
                        !mbar_wait_bounded(&tempty[buf], tphase ^ 1u, a.wait_limit, a.status, abort)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const int nk = min(GRP, a.kt - g * GRP);
                    for (int i = 0; i < nk; ++i) {
                        const uint64_t wd = d0 + (uint64_t)((stage * stage_bytes + i * w_bytes) >> 4);
                        const uint64_t ad = d0 + (uint64_t)((stage * stage_bytes + GRP * w_bytes + i * a_bytes) >> 4);
                        const uint32_t dt = tmem + (uint32_t)(buf * BUF_COLS + i * COLS);
                        tc::mma_f8(dt, ad, wd, idesc, 0u);
                        tc::mma_f8(dt, ad + 2, wd + 2, idesc, 1u);
                        tc::mma_f8(dt, ad + 4, wd + 4, idesc, 1u);
                        tc::mma_f8(dt, ad + 6, wd + 6, idesc, 1u);
                    }
                    tc::mma_commit(&tfull[buf]);        // a drain warp hands the stage back after this
                    if (++stage == a.stages) { stage = 0; phase ^= 1u; }
                    if (++buf == 2) { buf = 0; tphase ^= 1u; }
                }
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        // ---------------------------------------------------- drain warps
        const int ew = warp - CTRL_WARPS;
        const int quarter = warp & 3, half = ew >> 2;
        const int r = quarter * 32 + lane;                     // token row of the tile = TMEM lane
        pdl_wait();
        int buf = 0, stage = 0, parity = 0;
        uint32_t tphase = 0, xphase = 0;
        bool dead = false;
        for (int u = first; u < a.n_units; u += step) {
            int m0, n0;
            unit_rows(u, m0, n0);
            const int valid = min(BM, a.M - m0);
            const bool rv = r < valid;
            const bool live = quarter * 32 < valid;            // warp-uniform: some lane has a token
            const int col0 = n0 + half * HALF;                 // first weight-image row of this thread's columns
            // weight scales: plain, the blocks of the half's first column and the next one (16-column
            // piece p lies in the second where bit p of hi_mask is set); gated, gate and up of the unit's block
            const float *sw0, *sw1;
            uint32_t hi_mask = 0;
            if (GATED) {
                const int fb = min(n0 / (2 * QB), a.nblk - 1);
                sw0 = a.sw + (size_t)fb * a.kt;
                sw1 = sw0 + (size_t)a.nblk * a.kt;
            } else {
                const int b0 = col0 / QB;
                sw0 = a.sw + (size_t)min(b0, a.nblk - 1) * a.kt;
                sw1 = a.sw + (size_t)min(b0 + 1, a.nblk - 1) * a.kt;
#pragma unroll
                for (int p = 0; p < PPK; ++p) hi_mask |= ((col0 + 16 * p) / QB != b0) ? 1u << p : 0u;
            }
            float acc[HALF];
#pragma unroll
            for (int c = 0; c < HALF; ++c) acc[c] = 0.f;
            float nx[GRP] = {}, n0s[GRP] = {}, n1s[GRP] = {};  // scales of the next group, fetched one group ahead
            auto fetch = [&](int g) {
#pragma unroll
                for (int i = 0; i < GRP; ++i) {
                    const int kb = g * GRP + i;
                    const bool in = kb < a.kt;
                    nx[i] = in && rv ? load_sa(a, kb, m0 + r) : 0.f;
                    n0s[i] = in ? sw0[kb] : 0.f;
                    n1s[i] = in ? sw1[kb] : 0.f;
                }
            };
            if (live) fetch(0);
            for (int g = 0; g < n_grp; ++g) {
                float c0[GRP], c1[GRP];
#pragma unroll
                for (int i = 0; i < GRP; ++i) { c0[i] = nx[i] * n0s[i]; c1[i] = nx[i] * n1s[i]; }
                if (live && g + 1 < n_grp) fetch(g + 1);
                if (!dead && !mbar_wait_bounded(&tfull[buf], tphase, a.wait_limit, a.status, abort)) dead = true;
                dead = __any_sync(0xFFFFFFFFu, dead);          // warp-uniform: tcgen05.ld is warp-collective
                if (ew == 0 && lane == 0) mbar_arrive(&empty[stage]);
                if (!dead && live) {
                    tc::tc_fence_after();
                    const uint32_t tb = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * BUF_COLS + half * HALF);
                    auto col_of = [&](int j) -> uint32_t { return (uint32_t)((j / PPK) * COLS + (j % PPK) * 16); };
                    uint32_t pa[16], pb[16];
                    tc::tmem_ld16u(tb + col_of(0), pa);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t(&cur)[16] = (j & 1) ? pb : pa;
                        uint32_t(&nxt)[16] = (j & 1) ? pa : pb;
                        if (j < 7) tc::tmem_ld16u(tb + col_of(j + 1), nxt);
                        const int i = j / PPK, p = j % PPK;
                        if (g * GRP + i < a.kt) {
                            const float cl = GATED ? c0[i] : (((hi_mask >> p) & 1u) ? c1[i] : c0[i]);
                            const float ch = GATED ? c1[i] : cl;
#pragma unroll
                            for (int q = 0; q < 16; q += 2)
                                tc::fma2(acc[16 * p + q], acc[16 * p + q + 1], cur[q], cur[q + 1], q < 8 ? cl : ch);
                        }
                        if (j < 7) tc::tmem_wait_ld();
                    }
                    tc::tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[buf]);
                if (++buf == 2) { buf = 0; tphase ^= 1u; }
                if (++stage == a.stages) stage = 0;
            }

            if constexpr (GATED) {
                // piece p: 8 gate columns, then the same 8 features' up columns
                const int f0 = col0 / 2;                       // first feature of this thread
                float h[HALF / 2];
                float am = 0.f;
#pragma unroll
                for (int e = 0; e < HALF / 2; ++e) {
                    const float gt = acc[(e / 8) * 16 + (e % 8)], up = acc[(e / 8) * 16 + 8 + (e % 8)];
                    h[e] = f0 + e < a.N ? silu_mul(gt, up) : 0.f;
                    am = max_nan(am, fabsf(h[e]));
                }
                amax_cta[half * BM + r] = am;
                named_bar_sync(1, EPI_WARPS * 32);
                am = max_nan(amax_cta[r], amax_cta[BM + r]);
                if (csize > 1) {
                    // every CTA sends its rows' amax to every CTA of the cluster (itself included); a
                    // peer is at most one unit ahead, so two slots are enough
                    float* slot = amax_all + parity * MAX_CLUSTER * BM;
                    if (half == 0) {
                        const uint32_t mine = smem_addr(slot + rank * BM + r), bar = smem_addr(&xbar[parity]);
                        if (r == 0) mbar_arrive_expect_tx(&xbar[parity], csize * BM * 4u);
                        for (uint32_t p = 0; p < csize; ++p) st_async_f32(map_to_rank(mine, p), am, map_to_rank(bar, p));
                    }
                    if (!dead && !mbar_wait_cluster(&xbar[parity], xphase, a.wait_limit, a.status, abort)) dead = true;
                    for (uint32_t p = 0; p < csize; ++p) am = max_nan(am, slot[p * BM + r]);
                    if (++parity == 2) { parity = 0; xphase ^= 1u; }
                }
                uint32_t held;
                const float sc = group_scale(am, a.e8m0, held);
                const float is = inv_scale(sc);
                if (rv && !dead) {
                    uint8_t* dst = a.hq + (int64_t)(m0 + r) * a.ld_hq + f0;
#pragma unroll
                    for (int e = 0; e < HALF / 2; e += 8) {
                        const uint32_t lo = pack4_e4m3(h[e] * is, h[e + 1] * is, h[e + 2] * is, h[e + 3] * is);
                        const uint32_t hi = pack4_e4m3(h[e + 4] * is, h[e + 5] * is, h[e + 6] * is, h[e + 7] * is);
                        if (f0 + e + 8 <= a.N) {
                            *reinterpret_cast<uint2*>(dst + e) = make_uint2(lo, hi);
                        } else {
#pragma unroll
                            for (int b = 0; b < 8; ++b)
                                if (f0 + e + b < a.N) dst[e + b] = (uint8_t)((b < 4 ? lo >> (8 * b) : hi >> (8 * (b - 4))) & 0xFFu);
                        }
                    }
                    const int fb = n0 / (2 * QB);
                    if (half == 0 && rank == 0) {
                        const int64_t at = (int64_t)fb * a.ld_hs + m0 + r;
                        if (a.e8m0) static_cast<uint8_t*>(a.hs)[at] = (uint8_t)held;
                        else static_cast<uint32_t*>(a.hs)[at] = held;
                    }
                }
                named_bar_sync(1, EPI_WARPS * 32);             // amax_cta is reused by the next unit
            } else if (live && !dead) {
                // 16 columns at a time through the warp's staging tile, so that a store
                // instruction covers whole 32-byte sectors of 8 rows
                float* stg = stg_all + (size_t)ew * 32 * STG_STRIDE;
#pragma unroll
                for (int p = 0; p < PPK; ++p) {
                    const int cb = col0 + 16 * p;
                    if (cb >= a.N || half * HALF + 16 * p >= a.bn) continue;     // warp-uniform
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<float4*>(stg + lane * STG_STRIDE + 4 * i) = make_float4(
                            acc[16 * p + 4 * i], acc[16 * p + 4 * i + 1], acc[16 * p + 4 * i + 2], acc[16 * p + 4 * i + 3]);
                    __syncwarp();
                    if (a.y_vec && cb + 16 <= a.N) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const int rr = 8 * t + (lane >> 2), c = 4 * (lane & 3);
                            const float4 v = *reinterpret_cast<const float4*>(stg + rr * STG_STRIDE + c);
                            const int row = quarter * 32 + rr;
                            if (row < valid) {
                                const int64_t at = (int64_t)(m0 + row) * a.ldy + cb + c;
                                if (a.y_f32) {
                                    *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = v;
                                } else {
                                    __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
                                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) =
                                        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
                                }
                            }
                        }
                    } else {
#pragma unroll 4
                        for (int t = 0; t < 16; ++t) {
                            const int rr = 2 * t + (lane >> 4), c = lane & 15, row = quarter * 32 + rr;
                            const float v = stg[rr * STG_STRIDE + c];
                            if (row < valid && cb + c < a.N) {
                                const int64_t at = (int64_t)(m0 + row) * a.ldy + cb + c;
                                if (a.y_f32) static_cast<float*>(a.y)[at] = v;
                                else static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
    if (GATED && csize > 1) cluster_sync();     // nobody leaves while a peer may still send to it
}

// ------------------------------------------------------------------ launch
struct Plan {
    int grp, bn, cluster, units, n_nt;
};

template <int GRP, bool GATED>
cudaError_t launch(const GemmCall& c, const Plan& p, Args& a, const CUtensorMap& map, cudaStream_t s) {
    a.stages = std::min(MAX_STAGES, RING_MAX / (GRP * (a.bn + a.a_rows) * 128));
    // 16 KB behind the ring: the last block's operand read of a short token tile ends inside it
    // (STG_BYTES + AMAX_BYTES + 1 KB lie there)
    static_assert(STG_BYTES + AMAX_BYTES >= BM * 128, "operand read past the ring");
    const int smem = 1024 + a.stages * GRP * (a.bn + a.a_rows) * 128 + STG_BYTES + AMAX_BYTES + 2 * BM * 4;
    cudaError_t e = ensure_smem_limit<fp8_gemm_kernel<GRP, GATED>>(SMEM_MAX);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    if (GATED && p.cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = p.cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    int slots = c.lin->num_sms;
    if (GATED && p.cluster > 1) {
        // clusters that fit at once (a cluster stays inside one GPC), asked once: every plan of
        // this kernel has the same cluster size and one CTA per SM
        static std::atomic<int> fit{0};
        slots = fit.load(std::memory_order_relaxed);
        if (slots == 0) {
            cfg.gridDim = dim3(c.lin->num_sms / p.cluster * p.cluster);
            e = cudaOccupancyMaxActiveClusters(&slots, fp8_gemm_kernel<GRP, GATED>, &cfg);
            if (e != cudaSuccess) return e;
            if (slots < 1) return cudaErrorInvalidConfiguration;
            fit.store(slots, std::memory_order_relaxed);
        }
    }
    cfg.gridDim = dim3(std::min(p.units, slots) * p.cluster);
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<GRP, GATED>, map, a);
}

inline cudaError_t encode_a(const GemmCall& c, int a_rows, CUtensorMap* map) {
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)c.lin->d.in_features, (cuuint64_t)c.M};
    const cuuint64_t strides[1] = {(cuuint64_t)c.ld_aq};
    const cuuint32_t box[2] = {128, (cuuint32_t)a_rows}, one[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(c.aq), dims, strides, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

inline Args base_args(const GemmCall& c) {
    Args a = {};
    const moe_linear* L = c.lin;
    a.w = L->w;
    a.sw = L->sw;
    a.sa = c.as;
    a.ld_sa = c.ld_as;
    a.M = c.M;
    a.N = L->d.out_features;
    a.kt = L->kt;
    a.rows_pad = L->rows_pad;
    a.nblk = (L->d.out_features + QB - 1) / QB;
    a.a_rows = c.M >= BM ? BM : (c.M + 7) / 8 * 8;
    a.e8m0 = L->d.scale_type == MOE_SCALE_E8M0;
    a.status = L->dev_status;
    a.wait_limit = L->wait_limit;
    return a;
}

}  // namespace dg
}  // namespace moe
