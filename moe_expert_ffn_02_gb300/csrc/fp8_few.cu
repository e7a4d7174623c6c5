// FP8 projections of few tokens (1 to 64), plain and gated: the weights are
// streamed once, by all SMs.
//
// Bound by HBM: a call reads the weights' bytes and almost nothing else.  So
// the weights are the MMA's 128-row operand and the tokens its 16, 32 or 64
// columns: an MMA takes about 36 cycles here however few columns it has (it
// reads its 128-row operand from shared memory), so 128 weight rows per MMA keep
// the tensor core far ahead of the copies, and each of the four lane quarters
// has its own warps to drain it.
//
// The weights are cut into tiles of R <= 128 rows and S ranges of K; the S CTAs
// of a tile form a cluster and add their partial sums through distributed
// shared memory, in rank order.  R and S follow from the weights' shape alone,
// and blocks are added in K order, so a token's result does not depend on how
// many others are in the batch.  One SM takes at most about 70 GB/s and 100 of
// them saturate HBM (measured with bulk copies alone: 64 CTAs 4.4 TB/s, 96 6.3,
// 112 6.7, 152 6.8); two CTAs per SM with short ranges also shorten the chain of a call.
//
// A stage is a group of G K blocks (R rows of weights, the tokens, their
// scales): waiting on or arriving at an mbarrier takes a warp about 150 cycles
// and issuing a tensor copy about 90, so narrow tiles need several blocks per
// hand-off.  Half the SM's shared memory and tensor memory at most: two CTAs fit,
// so the next call's weights are requested while this one ends, and a cluster of
// eight finds room beside others.
//
// fp32 scales: each stage has its own tensor-memory buffer, drained and scaled in
// registers as its MMAs end, block by block in K order.  The two warps of a lane
// quarter take half of the tokens each: 8, 16 or 32 sums a thread, which leaves
// the 96 registers that two CTAs per SM allow without spilling (64 sums a thread
// spilled, and with shared memory taking the L1, 64 tokens cost 90 us where 16
// took 17).
// e8m0 scales: the tensor core applies them (mxf8f6f4, block_scale; see the
// many-token form), the range accumulates in tensor memory and is read once; warps
// 2 and 3 lay out the scale factors.  Ranges of more than 64 blocks take the first
// form, whose sums are not a single chain of truncating MMAs.
//
// Measured: 1 x 2048 x 7168 4.35 us, 16 x 7168 x 4096 with e8m0 scales 6.8 (4.4 TB/s), 1 x 18432 x 7168 20.8 (6.4),
// gated 1 x 7168 x 2048 8.25 (3.6), 1 x 7168 x 18432 47 (5.6): what is left is the chain from the preceding kernel's end
// (tokens' way in, last block, join, about 2.5 us), in which only the next call's first stages are
// copied.
//
// Gated: a cluster holds the 256 interleaved gate/up rows of 128 features (two
// tiles of 128 rows, S ranges of K each), which is one quantisation group.
#include "fp8_gemm.cuh"

#include <cmath>

namespace moe {
namespace few {

using namespace dg;

constexpr int MAX_M = 64;
constexpr int ST_MAX = 8;                    // ring stages
constexpr int KR_MAX = 512;                  // K blocks per range, at most (weight scales kept in shared memory)
// 4 control warps and 8 drain warps, launched at 80 registers so that two CTAs fit: 128 x 48 + 256 x 96 = 384 x 80
constexpr int FEW_CTRL_REGS = 48, FEW_DRAIN_REGS = 96;

struct FewArgs {
    const float* sw;
    int M, N, kt, nblk;
    int R, S, G;                             // rows per tile, K ranges, K blocks per stage (1, 2 or 4)
    int a_rows, stages, kr, kr4;             // kr: blocks of the longest range; kr4: up to a multiple of 4
    int k_full;
    void* y;
    int64_t ldy;
    bool y_f32;
    uint8_t* hq;
    int64_t ld_hq;
    void* hs;
    int64_t ld_hs;
    uint32_t* status;
    uint32_t wait_limit;
    bool plant;                              // the first CTA issues all of its MMAs but the last ones
};

// Four fp32 into a CTA of the cluster, counted on that CTA's mbarrier.
__device__ __forceinline__ void st_async_4(uint32_t remote, const float* v, uint32_t remote_bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(remote),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
                 "r"(remote_bar)
                 : "memory");
}
// A named barrier that also tells every thread whether `mine` held in all of them.
__device__ __forceinline__ bool named_bar_and(int id, int threads, bool mine) {
    uint32_t all;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %3, 0;\n barrier.cta.red.and.pred p, %1, %2, q;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(all)
                 : "r"(id), "r"(threads), "r"((uint32_t)mine)
                 : "memory");
    return all != 0;
}
// (a0, a1) += (x0, x1) * s * (c0, c1), rounded as s * c and one fma each.
__device__ __forceinline__ void fma2s(float& a0, float& a1, uint32_t x0, uint32_t x1, float s, float c0, float c1) {
    asm("{\n .reg .b64 a, x, c, s;\n mov.b64 a, {%0, %1};\n mov.b64 x, {%2, %3};\n mov.b64 c, {%5, %6};\n mov.b64 s, {%4, %4};\n"
        " mul.rn.f32x2 c, c, s;\n fma.rn.f32x2 a, x, c, a;\n mov.b64 {%0, %1}, a;\n}"
        : "+f"(a0), "+f"(a1)
        : "r"(x0), "r"(x1), "f"(s), "f"(c0), "f"(c1));
}

constexpr int COLS = 256;                    // tensor-memory columns of a CTA
// K blocks per stage, at most, and stages: each stage's accumulators have columns of their own.
constexpr int group_cap(int tn) { return tn == 64 ? 2 : 4; }
constexpr int tail_bytes(int tn) { return tn * BM * 4 > BM * 128 ? tn * BM * 4 : BM * 128; }   // partial sums; operand read

enum Mode { F32, E8, MX };                   // fp32 scales; e8m0 scales applied in registers; by the tensor core
constexpr int MX_MAX_KB = 64;                // K blocks of one accumulation chain
constexpr int MX_QUADS = MX_MAX_KB / 4;
constexpr int MX_SF_COL = 64;                // scale factors: columns 64 + 8 q, weights' then tokens'

// First K block of range p: ranges start at even blocks, whatever G is.
__host__ __device__ inline int range_start(int kt, int S, int p) { return p == S ? kt : (kt + 1) / 2 * p / S * 2; }

// Scales of 4 tokens of a K block's run.
template <bool E8>
__device__ __forceinline__ float4 load_sa4(const uint8_t* sl, int t, int a_rows) {
    const int to = min(t, a_rows - 4);         // a multiple of 4; tokens past a_rows are nobody's
    if constexpr (!E8) return *reinterpret_cast<const float4*>(sl + 4 * to);
    const uint32_t v = *reinterpret_cast<const uint32_t*>(sl + to);
    return make_float4(e8m0_to_f32((uint8_t)v), e8m0_to_f32((uint8_t)(v >> 8)), e8m0_to_f32((uint8_t)(v >> 16)),
                       e8m0_to_f32((uint8_t)(v >> 24)));
}

__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// acc[t] += D[t] * (s_w * s_x[t]) for HT tokens from t0 of KBS K blocks, TN columns apart in tensor
// memory.  Straight-line code from the loads to the products: the shared-memory reads of the scales
// overlap the tensor-memory loads, which a branch between would prevent.
template <int TN, int KBS, bool E8>
__device__ __forceinline__ void take(uint32_t tb, const uint8_t* sl, int pitch, const float* sw, int t0, int a_rows,
                                     float (&acc)[TN / 2]) {
    constexpr int HT = TN / 2, PC = HT < 16 ? HT : 16;
#pragma unroll
    for (int p = 0; p < HT; p += PC) {
        uint32_t raw[KBS][PC];
#pragma unroll
        for (int j = 0; j < KBS; ++j) {
            if constexpr (PC == 8) ld8(tb + j * TN, raw[j]);
            else tc::tmem_ld16u(tb + j * TN + p, raw[j]);
        }
        float4 c[KBS][PC / 4];
        float s[KBS];
#pragma unroll
        for (int j = 0; j < KBS; ++j) {
            s[j] = sw[2 * j];
#pragma unroll
            for (int q = 0; q < PC / 4; ++q) c[j][q] = load_sa4<E8>(sl + j * pitch, t0 + p + 4 * q, a_rows);
        }
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < KBS; ++j)
#pragma unroll
            for (int q = 0; q < PC / 4; ++q) {
                const int t = p + 4 * q;
                fma2s(acc[t], acc[t + 1], raw[j][4 * q], raw[j][4 * q + 1], s[j], c[j][q].x, c[j][q].y);
                fma2s(acc[t + 2], acc[t + 3], raw[j][4 * q + 2], raw[j][4 * q + 3], s[j], c[j][q].z, c[j][q].w);
            }
    }
}

__device__ __forceinline__ void store_y(const FewArgs& a, int t, int n, float v) {
    const int64_t at = (int64_t)t * a.ldy + n;
    if (a.y_f32) static_cast<float*>(a.y)[at] = v;
    else static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
}

template <int TN, bool GATED, Mode MODE>
__global__ void __launch_bounds__(NTHREADS, 2) few_kernel(const __grid_constant__ Maps maps, FewArgs a) {
    constexpr bool E8S = MODE != F32;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int w_bytes = a.R * 128, a_bytes = a.a_rows * 128, stage_bytes = a.G * (w_bytes + a_bytes);
    const int pitch = sa_pitch(a.a_rows, E8S), slot_bytes = (a.G * pitch + 127) / 128 * 128;
    uint8_t* recv = ring + a.stages * stage_bytes;                                  // [own token group][rank][row][4 tokens] fp32
    uint8_t* scales = recv + tail_bytes(TN);                                        // [stage][slot]; MX: [kr4][pitch]
    float* sws = reinterpret_cast<float*>(scales + a.stages * slot_bytes);          // [kr][2]
    uint8_t* packed = scales + (a.kr4 * pitch + 127) / 128 * 128;                   // MX: [quad][weights 512 B | tokens 512 B]
    __shared__ uint64_t full[ST_MAX], empty[ST_MAX], tfull[ST_MAX], sfull, sready[MODE == MX ? MX_QUADS : 1], joined, mma_done;
    __shared__ __align__(16) float amax[GATED ? 2 : 1][2][4][4];                                  // [parity][half of the threads][warp][token]
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int csize = GATED ? 2 * a.S : a.S;
    const int rank = (int)blockIdx.x % csize, unit = (int)blockIdx.x / csize;
    const int n0 = (GATED ? 2 * unit + rank / a.S : unit) * a.R;
    const int kb0 = range_start(a.kt, a.S, rank % a.S), nkb = range_start(a.kt, a.S, rank % a.S + 1) - kb0;
    const int n_grp = (nkb + a.G - 1) / a.G;
    const int pre = min(a.stages, n_grp);
    // groups of 4 tokens go to the cluster's CTAs in turn; this one finishes `own` of them
    const int own = csize > 1 ? ((a.M + 3) / 4 + csize - 1 - rank) / csize : 0;
    const uint32_t ring0 = smem_addr(ring), scl0 = smem_addr(scales), full0 = smem_addr(full);

    // a stage's bytes and the copy of its weights, by one thread
    auto copy_w = [&](int st, int g) {
        expect_tx(full0 + 8 * st, (uint32_t)(a.G * (w_bytes + (MODE == MX ? 0 : pitch)) +
                                             tokens_bytes(a.k_full, a.kt, kb0 + g * a.G, a.G, a_bytes)));
        tma_load_3d(ring0 + st * stage_bytes, &maps.w, 0, n0, kb0 + g * a.G, full0 + 8 * st);
    };

    pdl_trigger();
    if (threadIdx.x == 0) {
        const uint32_t drains = MODE == MX ? 1 : EPI_WARPS;
        for (int s = 0; s < a.stages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], drains); mbar_init(&tfull[s], 1); }
        mbar_init(&joined, 1);
        mbar_init(&mma_done, 1);
        if (MODE == MX) {
            mbar_init(&sfull, 1);
            for (int q = 0; q < (MODE == MX ? MX_QUADS : 1); ++q) mbar_init(&sready[q], 1);
        }
        fence_mbar_init();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        abort_flag = 0;
        if (own > 0) expect_tx(smem_addr(&joined), (uint32_t)(own * csize * a.R * 16));
        // the weights do not depend on the preceding kernel, nor on the rest of this one's set-up
        for (int g = 0; g < pre; ++g) copy_w(g, g);
    }
    __syncthreads();
    if (csize > 1) cluster_arrive();                           // waited for before anything is sent to a peer
    volatile int* abort = &abort_flag;

    if (warp < CTRL_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW_CTRL_REGS));
        if (warp == 0) {
            // ------------------------------------------------ producer
            const uint32_t el = elect_one();
            if (el) {
                prefetch_map(&maps.a);
                if (a.k_full < a.kt) prefetch_map(&maps.a_last);
                prefetch_map(&maps.s);
            }
            pdl_wait();
            if (MODE == MX && el) {                  // the range's token scales, all at once
                expect_tx(smem_addr(&sfull), (uint32_t)(a.kr4 * pitch));
                tma_load_2d(scl0, &maps.s, 0, kb0, smem_addr(&sfull));
            }
            int st = 0, g = 0;
            uint32_t phase = 0;
            for (; g < n_grp; ++g) {
                if (g >= pre) {
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[st], phase ^ 1u, a.wait_limit, a.status, abort))) break;
                    if (el) copy_w(st, g);
                }
                if (el) {
                    const uint32_t dst = ring0 + st * stage_bytes + a.G * w_bytes, bar = full0 + 8 * st;
                    const int kb = kb0 + g * a.G;
                    copy_tokens(maps, a.k_full, a.kt, dst, kb, a.G, 0, a_bytes, bar);
                    if (MODE != MX) tma_load_2d(scl0 + st * slot_bytes, &maps.s, 0, kb, bar);
                }
                __syncwarp();
                if (++st == a.stages) { st = 0; phase ^= 1u; }
            }
            for (int n = min(g, a.stages); n > 0; --n) {   // every issued copy lands before the CTA exits
                if (--st < 0) { st = a.stages - 1; phase ^= 1u; }
                mbar_wait_bounded(&full[st], phase, LANDING_LIMIT_US, a.status, nullptr);
            }
            if (MODE == MX) mbar_wait_bounded(&sfull, 0, LANDING_LIMIT_US, a.status, nullptr);
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issuer
            tc::tmem_alloc(&tmem_slot, COLS);
            tc::tc_fence_before();
            named_bar_sync(2, (1 + EPI_WARPS) * 32);
            tc::tc_fence_after();
            pdl_wait();                                        // no bounded wait before it: limits count this kernel's time alone
            const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_slot, 0);
            const uint32_t el = elect_one();
            const uint32_t idesc = (1u << 4) | ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
            const uint32_t d0 = (uint32_t)tc::sw128_desc(ring0), sf0 = smem_addr(packed);
            int st = 0;
            uint32_t phase = 0;
            bool ok = true, issued = false;
            const int stop = a.plant && blockIdx.x == 0 ? n_grp - 1 : -1;
            for (int g = 0; g < n_grp && ok; ++g) {
                // A stage's accumulators are free when the stage is: the warps that drained them handed
                // it back, and its next copies were issued after that.
                ok = g != stop && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[st], phase, a.wait_limit, a.status, abort));
                if (!ok) break;
                tc::tc_fence_after();
                issued = true;
                const int nk = min(a.G, nkb - g * a.G);
                uint32_t wd = d0 + (uint32_t)((st * stage_bytes) >> 4), td = wd + (uint32_t)((a.G * w_bytes) >> 4);
                uint32_t dt = tmem + (uint32_t)(st * a.G * TN);
                for (int i = 0; i < nk; ++i) {
                    if constexpr (MODE == MX) {
                        const int k = g * a.G + i, q = k >> 2;
                        const uint32_t sft = tmem + MX_SF_COL + 8 * q;
                        if ((k & 3) == 0) {
                            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&sready[q], 0, a.wait_limit, a.status, abort));
                            if (!ok) break;
                            sf_copy(sft, sf_desc(sf0 + q * 1024), el);
                            sf_copy(sft + 4, sf_desc(sf0 + q * 1024 + 512), el);
                        }
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            mma_mx(tmem, wd + 2 * s, td + 2 * s, idesc_mx(TN, k & 3), sft, sft + 4, (k | s) != 0, el);
                    } else {
                        mma_block(dt, wd, td, idesc, el);
                    }
                    wd += (uint32_t)(w_bytes >> 4);
                    td += (uint32_t)(a_bytes >> 4);
                    dt += TN;
                }
                if (!ok) break;
                if (el) {
                    if (MODE == MX) {
                        tc::mma_commit(&empty[st]);
                        if (g == n_grp - 1) tc::mma_commit(&tfull[0]);
                    } else {
                        tc::mma_commit(&tfull[st]);
                    }
                }
                __syncwarp();
                if (++st == a.stages) { st = 0; phase ^= 1u; }
            }
            if (!ok && issued) finish_mmas(&mma_done, el, a.status);
        } else if (MODE == MX) {
            // ------------------------------------------------ scale factors of every second quad of K blocks
            // 128 rows x 4 bytes in 512: row r at (r mod 32) * 16 + (r / 32) * 4, one byte per K block.
            // Weights: a tile lies in two scale blocks (plain) or has gate and up rows (gated), so a row's
            // word is one of two.
            const int b0 = GATED ? unit : n0 / QB;
            const float* s0 = a.sw + (size_t)min(b0, a.nblk - 1) * a.kt + kb0;
            const float* s1 = a.sw + (size_t)(GATED ? min(b0, a.nblk - 1) + a.nblk : min(b0 + 1, a.nblk - 1)) * a.kt + kb0;
            const int nq = (nkb + 3) / 4;
            for (int q = warp - 2; q < nq; q += 2) {
                const int kb = 4 * q + (lane & 3);
                // an fp32 power of two's exponent field is its e8m0 byte (NaN 255, 2^-127 0)
                const uint32_t e = kb < nkb ? __float_as_uint(((lane & 4) ? s1 : s0)[kb]) >> 23 : 127u;
                uint32_t w0 = 0, w1 = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    w0 |= __shfl_sync(0xFFFFFFFFu, e, b) << (8 * b);
                    w1 |= __shfl_sync(0xFFFFFFFFu, e, 4 + b) << (8 * b);
                }
                uint32_t v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 32 * j + lane;
                    v[j] = (GATED ? ((r >> 3) & 1) != 0 : (n0 + r) / QB != n0 / QB) ? w1 : w0;
                }
                *reinterpret_cast<uint4*>(packed + q * 1024 + lane * 16) = make_uint4(v[0], v[1], v[2], v[3]);
            }
            pdl_wait();
            bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&sfull, 0, a.wait_limit, a.status, abort));
            for (int q = warp - 2; q < nq && ok; q += 2) {
                uint32_t v[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint8_t* p = scales + 4 * q * pitch + min(32 * j + lane, pitch - 1);
                    v[j] = (uint32_t)p[0] | (uint32_t)p[pitch] << 8 | (uint32_t)p[2 * pitch] << 16 | (uint32_t)p[3 * pitch] << 24;
                }
                *reinterpret_cast<uint2*>(packed + q * 1024 + 512 + lane * 16) = make_uint2(v[0], v[1]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&sready[q]);
            }
        }
        __syncwarp();
        named_bar_sync(3, NTHREADS);
        if (warp == 1) {
            tc::tc_fence_after();
            tc::tmem_dealloc(tmem_slot, COLS);
        }
        if (csize > 1) {                                       // the drain warps' two cluster barriers below
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FEW_DRAIN_REGS));
    // -------------------------------------------------------- drain warps
    const int ew = warp - CTRL_WARPS, quarter = warp & 3, half = ew >> 2;
    const int row = quarter * 32 + lane;                       // weight row of the tile = TMEM lane
    const bool live = quarter * 32 < a.R;
    if (MODE != MX) {
        // the range's weight scales, two per block: plain, those of the tile's first scale block and
        // the next one; gated, gate and up
        const int b0 = GATED ? unit : n0 / QB;
        const float* s0 = a.sw + (size_t)min(b0, a.nblk - 1) * a.kt + kb0;
        const float* s1 = a.sw + (size_t)(GATED ? min(b0, a.nblk - 1) + a.nblk : min(b0 + 1, a.nblk - 1)) * a.kt + kb0;
        for (int i = threadIdx.x - CTRL_WARPS * 32; i < 2 * nkb; i += EPI_WARPS * 32)
            sws[i] = (i & 1) ? s1[i >> 1] : s0[i >> 1];
    }
    const int sel = GATED ? (row >> 3) & 1 : ((n0 + row) / QB != n0 / QB);
    named_bar_sync(2, (1 + EPI_WARPS) * 32);
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot + ((uint32_t)(quarter * 32) << 16);
    const int csize_log = 31 - __clz(csize);                   // csize is a power of two
    const uint32_t recv0 = smem_addr(recv), joined0 = smem_addr(&joined);
    // this row's sums of 4 tokens from t, to the CTA that finishes them
    auto send = [&](int t, const float* v) {
        const int g = t / 4, to = g & (csize - 1), slot = g >> csize_log;
        if (row < a.R)
            st_async_4(map_to_rank(recv0 + (uint32_t)(((slot * csize + rank) * a.R + row) * 16), to), v, map_to_rank(joined0, to));
    };
    if (csize > 1) cluster_wait();                             // the peers have set up their barriers
    pdl_wait();                                                // before the first bounded wait, and the first write
    if constexpr (MODE == MX) {
        const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&tfull[0], 0, a.wait_limit, a.status, abort));
        if (live && ok) {
            tc::tc_fence_after();
            // the two warps of a quarter take eight tokens in turn
            uint32_t raw[TN / 16][8];
#pragma unroll
            for (int j = 0; j < TN / 16; ++j) ld8(tmem + 8 * half + 16 * j, raw[j]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < TN / 16; ++j) {
                const int c = 8 * half + 16 * j;
                if (c >= a.M) break;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(raw[j][e]);
                if (!GATED && csize == 1) {
                    if (row < a.R && n0 + row < a.N) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (c + e < a.M) store_y(a, c + e, n0 + row, v[e]);
                    }
                } else {
                    send(c, v);
                    if (c + 4 < a.M) send(c + 4, v + 4);
                }
            }
        }
    } else {
        constexpr int HT = TN / 2;
        const int t0 = half * HT;                              // my first token
        const bool mine = live && t0 < a.M;                    // warp-uniform: tcgen05.ld is warp-collective
        float acc[HT];
#pragma unroll
        for (int t = 0; t < HT; ++t) acc[t] = 0.f;
        int st = 0;
        uint32_t phase = 0;
        bool dead = false;
        for (int g = 0; g < n_grp; ++g) {
            const int k0 = g * a.G, nk = min(a.G, nkb - k0);
            // the second wait returns at once: it makes the stage's scales visible here
            if (!dead) {
                dead = !__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&tfull[st], phase, a.wait_limit, a.status, abort) &&
                                                    mbar_wait_bounded(&full[st], phase, a.wait_limit, a.status, abort));
            }
            if (mine && !dead) {
                tc::tc_fence_after();
                const uint32_t tb = tmem + (uint32_t)(st * a.G * TN + t0);
                const uint8_t* sl = scales + st * slot_bytes;
                const float* sw = sws + 2 * k0 + sel;
                int i = 0;
                if constexpr (TN <= 32) {                      // two blocks' loads in flight where registers allow
#pragma unroll 1
                    for (; i + 2 <= nk; i += 2) take<TN, 2, E8S>(tb + i * TN, sl + i * pitch, pitch, sw + 2 * i, t0, a.a_rows, acc);
                }
#pragma unroll 1
                for (; i < nk; ++i) take<TN, 1, E8S>(tb + i * TN, sl + i * pitch, pitch, sw + 2 * i, t0, a.a_rows, acc);
                tc::tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            if (++st == a.stages) { st = 0; phase ^= 1u; }
        }
        // sums that are not whole go nowhere: the CTA that waits for them gives up too, and writes nothing
        if (live && !dead) {
#pragma unroll
            for (int t = 0; t < HT; t += 4) {
                if (t0 + t >= a.M) break;
                if (!GATED && csize == 1) {
                    if (row < a.R && n0 + row < a.N) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (t0 + t + e < a.M) store_y(a, t0 + t + e, n0 + row, acc[t + e]);
                    }
                } else {
                    send(t0 + t, acc + t);
                }
            }
        }
    }
    // -------------------------------------------------------- join the K ranges
    // The sums were sent as they were drained, 512 bytes a warp and instruction; each CTA waits for its
    // token groups' bytes and finishes them from its own shared memory.  (Leaving them at home, a cluster
    // barrier and loads from the peers took 5,400 cycles, with another barrier before anyone may leave:
    // 64 x 7168 x 2048 gated 17.5 us, 50 x 1040 x 1000 5.7.)
    tc::tc_fence_before();
    named_bar_sync(3, NTHREADS);
    if (csize == 1) return;
    cluster_arrive();                                          // everything sent
    const bool whole = own > 0 && __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&joined, 0, a.wait_limit, a.status, abort));
    // gated: all warps go through, because they meet at a barrier there, which also tells them whether any of
    // them gave up (each on its own look at the clock); then none stores
    if (GATED ? own > 0 : whole) {
        const int tid = threadIdx.x - CTRL_WARPS * 32, side = tid >> 7, i = tid & 127;   // 128 threads a group
        const float4* in = reinterpret_cast<const float4*>(recv);
        if constexpr (GATED) {
            // a thread takes a feature of four tokens
            const int ff = i & 63, r = (ff >> 3) * 16 + (ff & 7);
            const int base = (i >> 6) * a.S;                   // first rank of the tile with this feature
            const int f = unit * QB + i;
            int parity = 0;
            for (int slot = side; slot < own; slot += 2, parity ^= 1) {
                float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
#pragma unroll 4
                for (int p = 0; p < a.S; ++p) {
                    const float4* at = in + (slot * csize + base + p) * BM + r;
                    g = add4(g, at[0]);
                    u = add4(u, at[8]);
                }
                float h[4] = {silu_mul(g.x, u.x), silu_mul(g.y, u.y), silu_mul(g.z, u.z), silu_mul(g.w, u.w)}, am[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (f >= a.N) h[e] = 0.f;
                    am[e] = fabsf(h[e]);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) am[e] = max_nan(am[e], __shfl_xor_sync(0xFFFFFFFFu, am[e], o));
                }
                float (&all)[4][4] = amax[parity][side];
                if (lane == 0) *reinterpret_cast<float4*>(all[ew & 3]) = make_float4(am[0], am[1], am[2], am[3]);
                const bool store = named_bar_and(4 + side, 128, whole);
                const int t0 = 4 * (slot * csize + rank);
                // lane e mod 4 works out token e's scale
                const int q = lane & 3;
                uint32_t held;
                const float is = inv_scale(group_scale(max_nan(max_nan(all[0][q], all[1][q]), max_nan(all[2][q], all[3][q])), E8S, held));
                uint8_t code[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) code[e] = (uint8_t)f32x2_to_e4m3x2(h[e] * __shfl_sync(0xFFFFFFFFu, is, e), 0.f);
                uint8_t* dst = a.hq + (int64_t)t0 * a.ld_hq + f;
#pragma unroll
                for (int e = 0; e < 4; ++e, dst += a.ld_hq)
                    if (store && t0 + e < a.M && f < a.N) *dst = code[e];
                if (store && i < 4 && t0 + i < a.M) {
                    const int64_t at = (int64_t)unit * a.ld_hs + t0 + i;
                    if (E8S) static_cast<uint8_t*>(a.hs)[at] = (uint8_t)held;
                    else static_cast<uint32_t*>(a.hs)[at] = held;
                }
            }
        } else {
            // a thread takes a row of four tokens
            for (int slot = side; slot < own; slot += 2) {
                if (i >= a.R || n0 + i >= a.N) break;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int p = 0; p < a.S; ++p) v = add4(v, in[(slot * csize + p) * a.R + i]);
                const int t0 = 4 * (slot * csize + rank);
                const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t0 + e < a.M) store_y(a, t0 + e, n0 + i, y[e]);
            }
        }
    }
    cluster_wait();                                            // nobody leaves while a peer may still send to it
    let_land(abort);
}

struct FewPlan {
    int R, S, G;
};

// The longest of S ranges of kt blocks.
static int longest_range(int kt, int S) {
    int kr = 0;
    for (int i = 0; i < S; ++i) kr = std::max(kr, range_start(kt, S, i + 1) - range_start(kt, S, i));
    return kr;
}

// Rows per tile and K ranges, from the weights' shape alone.  The weights of the estimate are fitted to
// which of the measured R and S is fastest (12 shapes, both scale types, 1, 20 and 64 tokens: within 1 % of
// the best on average), not to the times: a K block's MMAs and hand-offs, an SM's 70 GB/s, all SMs'
// 6.8 TB/s, a fixed cost per tile, per joined range and per CTA.  Short ranges win: 2048 x 7168, one token, takes
// 4.3 us with R = 128, S = 4 (224 CTAs) and 5.4 with R = 96, S = 2; 7168 x 4096, 64 tokens, 11.6 with R = 128,
// S = 8 and 15.2 with R = 64, S = 4.  Clusters do not pack every SM: past 92 % of the slots a second wave
// starts (7168 x 7168: 300 CTAs in clusters of four 12.1 us, 256 10.3).
static FewPlan plan_few(const moe_linear* L) {
    const bool gated = L->d.gated != 0;
    FewPlan best = {};
    double best_us = 0;
    const double slots = 2.0 * L->num_sms;
    for (int S = 1; S <= (gated ? 4 : 8); S *= 2) {
        if (S > (L->kt + 1) / 2) break;                        // every range holds a pair of blocks
        const int kr = longest_range(L->kt, S);
        if (kr > KR_MAX) continue;
        for (int R = gated ? BM : 16; R <= BM; R += 16) {
            const double tiles = gated ? 2.0 * ((L->d.out_features + QB - 1) / QB) : (double)((L->rows + R - 1) / R);
            const double ctas = tiles * S, per_sm = ctas <= L->num_sms ? 1.0 : 2.0;
            const double rounds = std::ceil(ctas / (gated || S > 1 ? 0.92 * slots : slots));
            const double cta = rounds * std::max(kr * (0.5 + 0.0013 * R), per_sm * kr * R * 128.0 / 70e3) + 1.2;
            const double hbm = L->kt * tiles * R * 128.0 / 6.8e6;
            const double us = std::sqrt(cta * cta + hbm * hbm) + (S > 1 ? 1.0 : 0.0) + 0.007 * ctas;
            if (!best.R || us < best_us) {
                best_us = us;
                best = FewPlan{R, S, R <= 64 && kr >= 8 ? 4 : 2};
            }
        }
    }
    return best;
}

template <int TN, bool GATED, Mode MODE>
cudaError_t launch_few(const GemmCall& c, const FewPlan& p, int kr, cudaStream_t s) {
    const moe_linear* L = c.lin;
    Args g = base_args(c);                    // what the tensor maps are made from
    g.bn = p.R;
    FewArgs a = {};
    a.sw = L->sw;
    a.M = c.M; a.N = L->d.out_features; a.kt = L->kt; a.nblk = g.nblk;
    a.R = p.R; a.S = p.S;
    a.a_rows = g.a_rows;
    a.kr = kr;
    a.kr4 = (kr + 3) / 4 * 4;
    a.k_full = g.k_full;
    a.y = c.y; a.ldy = c.ldy; a.y_f32 = c.y_f32;
    a.hq = c.hq; a.ld_hq = c.ld_hq; a.hs = c.hs; a.ld_hs = c.ld_hs;
    a.status = L->dev_status; a.wait_limit = L->wait_limit; a.plant = c.plant;
    // blocks per stage: the plan's, unless fewer than three stages would fit (one block: two)
    const int pitch = sa_pitch(a.a_rows, MODE != F32);
    int smem = 0;
    for (a.G = std::min(p.G, group_cap(TN)); a.G >= 1; a.G /= 2) {
        const int fixed = 1024 + tail_bytes(TN) + (MODE == MX ? (a.kr4 * pitch + 127) / 128 * 128 + a.kr4 / 4 * 1024 : kr * 8);
        const int stage = a.G * (p.R + a.a_rows) * 128 + (MODE == MX ? 0 : (a.G * pitch + 127) / 128 * 128);
        a.stages = std::min(ST_MAX, (SMEM_HALF - fixed) / stage);
        if (MODE != MX) a.stages = std::min(a.stages, COLS / (a.G * TN));
        a.stages = std::min(a.stages, (kr + a.G - 1) / a.G);
        smem = fixed + a.stages * stage;
        if (a.stages >= std::min(a.G == 1 ? 2 : 3, (kr + a.G - 1) / a.G)) break;
    }
    if (a.G < 1) return cudaErrorInvalidValue;
    Maps maps;                                // MX: the tokens' scales of a whole range in one copy
    if (!encode_maps(c, g, a.G, MODE == F32 ? a.a_rows : pitch, MODE == MX ? a.kr4 : a.G, &maps)) return cudaErrorInvalidValue;
    cudaError_t e = ensure_smem_limit<few_kernel<TN, GATED, MODE>>(SMEM_HALF);
    if (e != cudaSuccess) return e;
    const int cluster = GATED ? 2 * p.S : p.S;
    const int tiles = GATED ? (L->d.out_features + QB - 1) / QB : (L->rows + p.R - 1) / p.R;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)(tiles * cluster));
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, few_kernel<TN, GATED, MODE>, maps, a);
}

template <bool GATED, Mode MODE>
static cudaError_t launch_tokens(const GemmCall& c, const FewPlan& p, int kr, cudaStream_t s) {
    if (c.M <= 16) return launch_few<16, GATED, MODE>(c, p, kr, s);
    if (c.M <= 32) return launch_few<32, GATED, MODE>(c, p, kr, s);
    return launch_few<64, GATED, MODE>(c, p, kr, s);
}

template <bool GATED>
static cudaError_t launch_mode(const GemmCall& c, cudaStream_t s) {
    const FewPlan p = {c.lin->few_R, c.lin->few_S, c.lin->few_G};
    const int kr = longest_range(c.lin->kt, p.S);
    if (c.lin->d.scale_type == MOE_SCALE_F32) return launch_tokens<GATED, F32>(c, p, kr, s);
    return kr <= MX_MAX_KB ? launch_tokens<GATED, MX>(c, p, kr, s) : launch_tokens<GATED, E8>(c, p, kr, s);
}

}  // namespace few

void plan_fp8_few(moe_linear* L) {
    const few::FewPlan p = few::plan_few(L);
    L->few_R = p.R;
    L->few_S = p.S;
    L->few_G = p.G;
}

bool few_tokens(const GemmCall& c) { return c.M <= few::MAX_M && c.lin->few_R != 0; }

cudaError_t launch_fp8_few(const GemmCall& c, bool gated, cudaStream_t s) {
    return gated ? few::launch_mode<true>(c, s) : few::launch_mode<false>(c, s);
}

}  // namespace moe
