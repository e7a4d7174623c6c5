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
// This form takes 65 tokens and more.  128 tokens are the MMA's M (TMEM lanes), BN weight rows its N
// (TMEM columns): a lane is one token, so sa is a per-thread scalar and sw uniform per 16 columns.  BN
// is a multiple of 16 chosen per call: narrow tiles give every SM a share of the weights,
// BN = 256 reuses the tokens best.
//
// A TMEM buffer holds 256 columns: GRP = 1, 2, 4 or 8 K blocks of up to
// 256 / GRP columns, which are also one stage of the copy ring.  One commit
// covers the group, because a commit costs about 512 cycles of MMA time however
// little work it closes: narrow tiles need several blocks per commit.  Drain
// warp (quarter, half) owns 32 lanes and the half's columns of every block of
// the group, so blocks are added in K order into the same accumulators whatever BN is.
//
// Warps: 0 copies (TMA), 1 issues the MMAs, 2 and 3 idle, 4-11 drain; the drain
// warps fetch the scales themselves, two groups ahead.  Token tiles with fewer
// than 128 rows copy only those rows (rounded up to 8); the MMA reads whatever lies
// behind them in shared memory into TMEM lanes nobody reads.
//
// Copies of weights start before the wait for the preceding kernel, and before
// the tensor memory is allocated.
//
// Where tiles alone leave SMs idle, a cluster of S CTAs shares each tile's K and
// adds the partial sums through distributed shared memory (BN = 128 and 256).
//
// Bound, many tokens: a 256-row block's MMAs take 512 cycles, its draining and
// scaling with the hand-offs round it about 780 (two buffers, eight warps).  8192 tokens: 2048 x 7168 105 us
// (2.3 PFLOP/s; the tensor pipe busy 47 % of the time), gated 7168 x 2048 196 us (2.45; 51 %).  Some hundreds
// of tokens: the copies into an SM, about 118 GB/s (777 x 1992 x 1001: 8.1 us).
#pragma once
#include "dense_internal.cuh"
#include "tcgen05.cuh"

#include <algorithm>
#include <cmath>

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
// What lies behind the ring: the plain epilogue's staging tiles (4 KB a warp where the copy engine
// writes the rows), or the gated one's amax of each half and, behind it, its amax exchange or its
// staging tiles (2 KB a warp); at least the 16 KB that the last block's 128-row operand read may run
// into.
constexpr int TMA_STG = 4096, CODE_STG = 2048;
constexpr int TAIL_PLAIN = STG_BYTES, TAIL_PLAIN_TMA = EPI_WARPS * TMA_STG;
constexpr int AMAX_CTA = 2 * BM * 4, TAIL_GATED = AMAX_CTA + EPI_WARPS * CODE_STG;
static_assert(TAIL_PLAIN >= BM * 128 && TAIL_GATED >= BM * 128 && AMAX_BYTES + AMAX_CTA <= TAIL_GATED, "tail");
constexpr int tail_bytes(int grp, bool gated) { return gated ? TAIL_GATED : grp == 1 ? TAIL_PLAIN_TMA : TAIL_PLAIN; }
// Bytes of one K block's token scales in shared memory (few-token form).
__host__ __device__ inline int sa_pitch(int a_rows, bool e8m0) { return e8m0 ? (a_rows + 15) / 16 * 16 : a_rows * 4; }
// Bytes of a stage: GRP blocks of operands.
inline int stage_cost(int grp, int bn, int a_rows) { return grp * (bn + a_rows) * 128; }
inline int ring_max() { return SMEM_MAX - 1024 - TAIL_PLAIN; }         // plain
// Shared memory of a CTA that leaves room for a second one on the SM.
constexpr int SMEM_HALF = 113 * 1024 - 2048;

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
    int S;                    // K ranges of a unit, one per CTA of its cluster; 1: none
    bool e8m0;
    int k_full;               // whole K blocks: K / 128; a ragged last one is copied on its own
    // plain
    void* y;
    int64_t ldy;
    bool y_f32, y_vec, y_wide; // y_vec: four columns a store; y_wide: eight, bf16
    bool y_tma;                // rows on 16-byte strides, written by the copy engine
    // gated
    uint8_t* hq;
    int64_t ld_hq;
    void* hs;
    int64_t ld_hs;
    uint32_t* status;
    uint32_t wait_limit;
    bool plant;                // the first CTA issues all MMAs of its first tile but the last ones
};

// What TMA brings: token codes (whole K blocks, and a ragged last one), weight image, token scales.
// What it takes: y, 32 rows of 128 bytes at a time.
struct Maps {
    CUtensorMap a, a_last, w, s, y;
};

__device__ __forceinline__ uint32_t idesc_for(int n) {   // D f32, A = B = E4M3, K-major, M = 128
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

// True in one lane of a converged warp.  The loops around it stay warp-uniform, so that
// descriptors and addresses live in uniform registers and an issue costs a few cycles.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n cp.async.bulk.commit_group;" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
}
// This thread's stores have read shared memory; have written memory.
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Token tiles of n K blocks from kb, rows m0.., one after the other at dst: one copy, or block by
// block where the ragged last one is among them.  Bytes that arrive: tokens_bytes.
__device__ __forceinline__ void copy_tokens(const Maps& m, int k_full, int kt, uint32_t dst, int kb, int n, int m0, int a_bytes, uint32_t bar) {
    if (k_full == kt || kb + n <= k_full) {
        tma_load_3d(dst, &m.a, 0, m0, kb, bar);
        return;
    }
    for (int i = 0; i < n && kb + i < kt; ++i) tma_load_3d(dst + i * a_bytes, &m.a_last, (kb + i) * QB, m0, 0, bar);
}
__device__ __forceinline__ int tokens_bytes(int k_full, int kt, int kb, int n, int a_bytes) {
    return (k_full == kt || kb + n <= k_full ? n : min(n, kt - kb)) * a_bytes;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// The four K32 steps of a block's MMA, by the elected lane.  lo: low words of the operands'
// descriptors; a K step of 32 bytes inside the swizzle atom adds 2.
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t a_lo, uint32_t w_lo, uint32_t idesc, uint32_t elected) {
    constexpr uint32_t HI = (uint32_t)(tc::DESC_HI >> 32);
    asm volatile(
        "{\n .reg .pred q, t;\n .reg .b64 a, w;\n .reg .b32 x, y;\n"
        " setp.ne.b32 q, %5, 0;\n setp.ne.b32 t, 0, 0;\n"
        " mov.b64 a, {%1, %4};\n mov.b64 w, {%2, %4};\n"
        " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, w, %3, t;\n"
        " setp.eq.b32 t, 0, 0;\n"
        " add.u32 x, %1, 2;\n add.u32 y, %2, 2;\n mov.b64 a, {x, %4};\n mov.b64 w, {y, %4};\n"
        " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, w, %3, t;\n"
        " add.u32 x, %1, 4;\n add.u32 y, %2, 4;\n mov.b64 a, {x, %4};\n mov.b64 w, {y, %4};\n"
        " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, w, %3, t;\n"
        " add.u32 x, %1, 6;\n add.u32 y, %2, 6;\n mov.b64 a, {x, %4};\n mov.b64 w, {y, %4};\n"
        " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, w, %3, t;\n}" ::"r"(d),
        "r"(a_lo), "r"(w_lo), "r"(idesc), "n"(HI), "r"(elected)
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
// Relaxed: after mbarrier.init and its own fence.  Releasing: orders this thread's accesses to its
// peers' shared memory before the arrival.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_release() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
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

// For an issuer that stopped early: the MMAs and scale copies that it has issued finish, before tensor memory is
// freed and the CTA leaves.
__device__ __forceinline__ void finish_mmas(uint64_t* done, uint32_t elected, uint32_t* status) {
    if (elected) tc::mma_commit(done);
    __syncwarp();
    mbar_wait_bounded(done, 0, LANDING_LIMIT_US, status, nullptr);
}

// After a cluster's last barrier, in a CTA that gave up: what its peers sent before they arrived there (a store into
// a peer's shared memory takes about a microsecond) lands before that memory is given back.  A CTA that did not give
// up has waited for every byte.
__device__ __forceinline__ void let_land(volatile int* abort) {
    if (*abort != 0)
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// ------------------------------------------------------------------ scaling by the tensor core
// Descriptor of a scale-factor block: no swizzle, 8-row groups of 128 bytes one after the other.
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint64_t desc, uint32_t elected) {
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n @q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}" ::"r"(taddr),
                 "l"(desc), "r"(elected)
                 : "memory");
}

// One K32 step with scale factors.
__device__ __forceinline__ void mma_mx(uint32_t d, uint32_t a_lo, uint32_t w_lo, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate, uint32_t elected) {
    constexpr uint32_t HI = (uint32_t)(tc::DESC_HI >> 32);
    asm volatile(
        "{\n .reg .pred q, t;\n .reg .b64 a, w;\n"
        " setp.ne.b32 q, %8, 0;\n setp.ne.b32 t, %7, 0;\n"
        " mov.b64 a, {%1, %4};\n mov.b64 w, {%2, %4};\n"
        " @q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, w, %3, [%5], [%6], t;\n}" ::"r"(d),
        "r"(a_lo), "r"(w_lo), "r"(idesc), "n"(HI), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(elected)
        : "memory");
}

// Instruction descriptor, kind::mxf8f6f4: A = B = E4M3, K-major, UE8M0 scales, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_mx(int n, int sf_id) {
    return ((uint32_t)sf_id << 4) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(BM >> 4) << 24) | ((uint32_t)sf_id << 29);
}

// One look at a barrier; unlike try_wait it never suspends the thread.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Batch b of a thread's accumulator columns: PIECE consecutive ones of the sequence
// (K block of the group, column of the half).
template <int HALF, int COLS, int PIECE>
__device__ __forceinline__ void ld_batch(uint32_t tb, int b, uint32_t (&raw)[PIECE]) {
    constexpr int W = HALF < 32 ? 16 : 32;
#pragma unroll
    for (int t = 0; t < PIECE; t += W) {
        const int seq = b * PIECE + t;
        const uint32_t at = tb + (uint32_t)((seq / HALF) * COLS + seq % HALF);
        if constexpr (W == 32) tc::tmem_ld32u(at, reinterpret_cast<uint32_t(&)[32]>(raw[t]));
        else tc::tmem_ld16u(at, reinterpret_cast<uint32_t(&)[16]>(raw[t]));
    }
}

// ------------------------------------------------------------------ epilogues
// One drain warp's place in the tile, and what the warps of the CTA (and cluster) share.
struct EpiCtx {
    int ew, quarter, half, lane;
    uint32_t rank, csize;
    uint8_t* stg;                  // the warp's staging tile: 32 rows of STG_STRIDE floats, 128 bytes (TMA) or 64 codes
    float* amax_cta;               // gated: [half][128]
    float* amax_all;               // gated: [parity][rank][128]
    uint64_t* xbar;                // gated: [parity]
    int parity;
    uint32_t xphase;
    volatile int* abort;
};

template <bool TMA>
__device__ __forceinline__ uint8_t* staging(uint8_t* tail, bool gated, int ew) {
    return gated ? tail + AMAX_CTA + ew * CODE_STG : tail + ew * (TMA ? TMA_STG : 32 * STG_STRIDE * 4);
}

// h = SiLU(g) * u of this thread's row and features, and its 1x128 E4M3 codes.  acc: pieces of 8
// gate columns and the same 8 features' up columns.
template <int HALF>
__device__ __forceinline__ void epi_gated(const Args& a, EpiCtx& x, const float (&acc)[HALF], int m0, int n0, int valid,
                                          bool& dead) {
    const int r = x.quarter * 32 + x.lane;
    const int f0 = (n0 + x.half * HALF) / 2;                   // first feature of this thread
    float h[HALF / 2];
    float am = 0.f;
    // no test per feature: a branch round each SiLU serialises their chains (106 cycles a feature instead of 32)
#pragma unroll
    for (int e = 0; e < HALF / 2; ++e) h[e] = silu_mul(acc[(e / 8) * 16 + (e % 8)], acc[(e / 8) * 16 + 8 + (e % 8)]);
    if (f0 + HALF / 2 > a.N) {                                 // warp-uniform
#pragma unroll
        for (int e = 0; e < HALF / 2; ++e)
            if (f0 + e >= a.N) h[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < HALF / 2; ++e) am = max_nan(am, fabsf(h[e]));
    x.amax_cta[x.half * BM + r] = am;
    named_bar_sync(1, EPI_WARPS * 32);
    am = max_nan(x.amax_cta[r], x.amax_cta[BM + r]);
    // a warp that gave up has no whole sums, and its amax belongs to all of the row's codes: after it the CTA neither
    // stores nor sends, so that the waits of its peers expire too and nobody's scales follow a part of a row
    dead = dead || *x.abort != 0;
    if (x.csize > 1) {
        // every CTA sends its rows' amax to every CTA of the cluster (itself included); a peer is
        // at most one unit ahead, so two slots are enough
        float* slot = x.amax_all + x.parity * MAX_CLUSTER * BM;
        if (x.half == 0 && !dead) {
            const uint32_t mine = smem_addr(slot + x.rank * BM + r), bar = smem_addr(&x.xbar[x.parity]);
            if (r == 0) mbar_arrive_expect_tx(&x.xbar[x.parity], x.csize * BM * 4u);
            for (uint32_t p = 0; p < x.csize; ++p) st_async_f32(map_to_rank(mine, p), am, map_to_rank(bar, p));
        }
        if (!dead && !mbar_wait_cluster(&x.xbar[x.parity], x.xphase, a.wait_limit, a.status, x.abort)) dead = true;
        for (uint32_t p = 0; p < x.csize; ++p) am = max_nan(am, slot[p * BM + r]);
        if (++x.parity == 2) { x.parity = 0; x.xphase ^= 1u; }
    }
    uint32_t held;
    // h / s as h * (1 / s): within one ulp of the quotient, far inside the code spacing
    const float is = inv_scale(group_scale(am, a.e8m0, held));
    uint32_t w[HALF / 8];
#pragma unroll
    for (int e = 0; e < HALF / 2; e += 4) w[e / 4] = pack4_e4m3(h[e] * is, h[e + 1] * is, h[e + 2] * is, h[e + 3] * is);
    // 64 codes a row go through the staging tile, so that a store covers them in 8 rows; its 16-byte
    // chunks are swizzled over the banks
    const bool staged = HALF == 128 && f0 + HALF / 2 <= a.N;   // warp-uniform
    if (staged && !dead) {
#pragma unroll
        for (int i = 0; i < HALF / 32; ++i)
            *reinterpret_cast<uint4*>(x.stg + x.lane * 64 + ((i ^ ((x.lane >> 1) & 3)) * 16)) =
                make_uint4(w[4 * i % (HALF / 8)], w[(4 * i + 1) % (HALF / 8)], w[(4 * i + 2) % (HALF / 8)], w[(4 * i + 3) % (HALF / 8)]);
        __syncwarp();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int rr = 8 * t + (x.lane >> 2), row = x.quarter * 32 + rr;
            const uint4 v = *reinterpret_cast<const uint4*>(x.stg + rr * 64 + (((x.lane & 3) ^ ((rr >> 1) & 3)) * 16));
            if (row < valid) *reinterpret_cast<uint4*>(a.hq + (int64_t)(m0 + row) * a.ld_hq + f0 + 16 * (x.lane & 3)) = v;
        }
    }
    if (r < valid && !dead) {
        uint8_t* dst = a.hq + (int64_t)(m0 + r) * a.ld_hq + f0;
        static_assert(HALF >= 32, "16 codes a store");         // rows start on 16 bytes
#pragma unroll
        for (int i = 0; i < HALF / 8 && !staged; i += 4) {
            if (f0 + 4 * (i + 4) <= a.N) {
                *reinterpret_cast<uint4*>(dst + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            } else {
#pragma unroll
                for (int b = 0; b < 16; ++b)
                    if (f0 + 4 * i + b < a.N) dst[4 * i + b] = (uint8_t)(w[i + b / 4] >> (8 * (b & 3)));
            }
        }
        if (x.half == 0 && x.rank == 0) {
            const int64_t at = (int64_t)(n0 / (2 * QB)) * a.ld_hs + m0 + r;
            if (a.e8m0) static_cast<uint8_t*>(a.hs)[at] = (uint8_t)held;
            else static_cast<uint32_t*>(a.hs)[at] = held;
        }
    }
    named_bar_sync(1, EPI_WARPS * 32);                         // amax_cta is reused by the next unit
}

// fp32 or bf16 rows: 16 columns at a time through the warp's staging tile, so that a store
// instruction covers whole 32-byte sectors of 8 rows.
template <int HALF, bool BIG>
__device__ __forceinline__ void epi_plain(const CUtensorMap& map_y, const Args& a, const EpiCtx& x, const float (&acc)[HALF], int m0, int n0, int valid) {
    const int row0 = x.quarter * 32, lane = x.lane;
    const int first = n0 + x.half * HALF;
    if (BIG && a.y_tma) {
        // 128 bytes of 32 rows at a time, handed to the copy engine: all CTAs finish their tiles at about
        // the same time, and the last piece's way to memory overlaps the next tile.  Columns and rows
        // past the end are clipped by the tensor map.  Swizzle: 16-byte chunk c of row r at c ^ (r mod 8).
        uint8_t* row = x.stg + lane * 128;
        const int per = a.y_f32 ? 32 : 64;
#pragma unroll
        for (int c0 = 0; c0 < HALF; c0 += 32) {
            const bool fresh = a.y_f32 || c0 % 64 == 0;
            if (fresh) {
                if (lane == 0) tma_store_read();
                __syncwarp();
            }
            if (a.y_f32) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<float4*>(row + ((j ^ (lane & 7)) * 16)) =
                        make_float4(acc[(c0 + 4 * j) % HALF], acc[(c0 + 4 * j + 1) % HALF], acc[(c0 + 4 * j + 2) % HALF],
                                    acc[(c0 + 4 * j + 3) % HALF]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        __nv_bfloat162 v = __floats2bfloat162_rn(acc[(c0 + 8 * j + 2 * k) % HALF], acc[(c0 + 8 * j + 2 * k + 1) % HALF]);
                        w[k] = *reinterpret_cast<uint32_t*>(&v);
                    }
                    *reinterpret_cast<uint4*>(row + (((j + (c0 / 32 % 2) * 4) ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (a.y_f32 || c0 % 64 == 32) {
                const int c = first + (c0 + 32 - per);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0 && c < a.N) tma_store_2d(&map_y, smem_addr(x.stg), c, m0 + row0);
            }
        }
        return;
    }
    if (a.y_wide && HALF >= 32 && first + HALF <= a.N && x.half * HALF + HALF <= a.bn) {
        // bf16, 32 columns at a time: a store covers 64 bytes of 8 rows, with half the instructions of the
        // 16-column form below (8192 x 2048 x 7168: 134 -> 118 us; e8m0 4096 x 7168 x 7168: 133.5 -> 132)
        uint8_t* st = x.stg;
        constexpr int PITCH = STG_STRIDE * 4;
#pragma unroll
        for (int c0 = 0; c0 < HALF; c0 += 32) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    __nv_bfloat162 v = __floats2bfloat162_rn(acc[(c0 + i + 2 * k) % HALF], acc[(c0 + i + 2 * k + 1) % HALF]);
                    w[k] = *reinterpret_cast<uint32_t*>(&v);
                }
                *reinterpret_cast<uint4*>(st + lane * PITCH + 2 * i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int rr = 8 * t + (lane >> 2);
                const uint4 v = *reinterpret_cast<const uint4*>(st + rr * PITCH + 16 * (lane & 3));
                if (row0 + rr < valid)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + (int64_t)(m0 + row0 + rr) * a.ldy + first + c0 + 8 * (lane & 3)) = v;
            }
            __syncwarp();
        }
        return;
    }
    float* stg = reinterpret_cast<float*>(x.stg);
    auto piece = [&](int p) {                                  // 16 columns
        const int cb = n0 + x.half * HALF + 16 * p;
        if (cb >= a.N || x.half * HALF + 16 * p >= a.bn) return;           // warp-uniform
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(stg + lane * STG_STRIDE + 4 * i) =
                make_float4(acc[16 * p + 4 * i], acc[16 * p + 4 * i + 1], acc[16 * p + 4 * i + 2], acc[16 * p + 4 * i + 3]);
        __syncwarp();
        if (a.y_vec && cb + 16 <= a.N) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int rr = 8 * t + (lane >> 2), c = 4 * (lane & 3);
                const float4 v = *reinterpret_cast<const float4*>(stg + rr * STG_STRIDE + c);
                if (row0 + rr < valid) {
                    const int64_t at = (int64_t)(m0 + row0 + rr) * a.ldy + cb + c;
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
            // rows or columns off the vector grid: two rows of 16 columns a store, eight loads ahead
#pragma unroll 1
            for (int t0 = 0; t0 < 16; t0 += 8) {
                float v[8];
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] = stg[(2 * (t0 + t) + (lane >> 4)) * STG_STRIDE + (lane & 15)];
                const int c = lane & 15;
                int64_t at = (int64_t)(m0 + row0 + 2 * t0 + (lane >> 4)) * a.ldy + cb + c;
#pragma unroll
                for (int t = 0; t < 8; ++t, at += 2 * a.ldy) {
                    if (row0 + 2 * (t0 + t) + (lane >> 4) < valid && cb + c < a.N) {
                        if (a.y_f32) static_cast<float*>(a.y)[at] = v[t];
                        else static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v[t]);
                    }
                }
            }
        }
        __syncwarp();
    };
    // bf16 rows that start at any element: words on the memory's four-byte grid, CH columns of a row (64 or 128
    // bytes) next to each other in a store; where a row's run starts inside a word, its first and last
    // element go on their own.  (998 x 145 x 6925: 12.1 us instead of 16.6 with two-byte stores, 8000 x 2000 x
    // 7001 132 instead of 162.)  fp32 rows off the vector grid, 256-row tiles: 32 columns the same way.
    constexpr int CH = BIG ? 64 : 32, W = CH / 2;
    uint32_t* words = reinterpret_cast<uint32_t*>(x.stg);      // [row][word j at j ^ (row mod W)]
#pragma unroll
    for (int c0 = 0; c0 < HALF; c0 += CH) {
        if (HALF < CH || (a.y_f32 && !BIG) || a.y_vec || first + c0 + CH > a.N || x.half * HALF + c0 + CH > a.bn) {
#pragma unroll
            for (int p = c0 / 16; p < (c0 + CH) / 16 && p < HALF / 16; ++p) piece(p);
            continue;
        }
        const int64_t at0 = (int64_t)(m0 + row0) * a.ldy + first + c0;
        if (BIG && a.y_f32) {
#pragma unroll
            for (int c = 0; c < CH; c += 32) {
                float* f = reinterpret_cast<float*>(words);
#pragma unroll
                for (int k = 0; k < 32; ++k) f[lane * 32 + (k ^ lane)] = acc[(c0 + c + k) % HALF];
                __syncwarp();
                float* y0 = static_cast<float*>(a.y) + at0 + c + lane;
#pragma unroll 8
                for (int rr = 0; rr < 32; ++rr, y0 += a.ldy) {
                    const float v = f[rr * 32 + (lane ^ rr)];
                    if (row0 + rr < valid) *y0 = v;
                }
                __syncwarp();
            }
            continue;
        }
        uint16_t* y0 = static_cast<uint16_t*>(a.y) + at0;
        const int odd0 = (int)(reinterpret_cast<uintptr_t>(y0) >> 1) & 1, step = (int)(a.ldy & 1);
        const bool odd = ((odd0 + lane * step) & 1) != 0;
        uint32_t last = 0;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            __nv_bfloat162 v = __floats2bfloat162_rn(acc[(c0 + 2 * k) % HALF], acc[(c0 + 2 * k + 1) % HALF]);
            const uint32_t now = *reinterpret_cast<uint32_t*>(&v);
            words[lane * W + (k ^ (lane & (W - 1)))] = odd ? __funnelshift_l(last, now, 16) : now;
            last = now;
        }
        if (odd && row0 + lane < valid) {
            __nv_bfloat16* mine = reinterpret_cast<__nv_bfloat16*>(y0 + lane * a.ldy);
            mine[0] = __float2bfloat16_rn(acc[c0 % HALF]);
            mine[CH - 1] = __float2bfloat16_rn(acc[(c0 + CH - 1) % HALF]);
        }
        __syncwarp();
#pragma unroll 8
        for (int t = 0; t < W; ++t) {
            const int rr = t * (32 / W) + lane / W, j = lane % W, o = (odd0 + rr * step) & 1;
            const uint32_t v = words[rr * W + (j ^ (rr & (W - 1)))];
            if (row0 + rr < valid && (o == 0 || j > 0)) *reinterpret_cast<uint32_t*>(y0 + rr * a.ldy - o + 2 * j) = v;
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ K ranges
// With S > 1 the CTAs of a cluster have a K range of the same unit each.  Every one leaves its
// partial sums in its shared memory, [128 rows][BN + 4] fp32 over the ring (one unit per cluster, so
// no copy is in flight any more); then the rows are dealt out, and a warp adds a row's S partials in
// rank order and finishes it.
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// Before the barrier after which the sums are joined: a warp that gave up raises the flags of all the cluster's
// CTAs, and none of them joins the unit.
__device__ __forceinline__ void tell_peers(bool dead, volatile int* abort, int ctas, int lane) {
    if (dead && lane < ctas)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(smem_addr(const_cast<int*>(abort)), (uint32_t)lane)), "r"(1u)
                     : "memory");
}

constexpr int part_pitch(int bn) { return bn + 4; }          // floats; 16-byte rows, free of bank conflicts

template <int HALF>
__device__ __forceinline__ void leave_partial(float* part, int half, int r, const float (&acc)[HALF]) {
    float* p = part + r * part_pitch(2 * HALF) + half * HALF;
#pragma unroll
    for (int c = 0; c < HALF; c += 4) *reinterpret_cast<float4*>(p + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
}

// The codes of 4 features from f (of the unit's 128) and, by lane 0, the group's scale, of R rows: one
// warp holds the rows' 128 features.  A row's way through SiLU, the largest of 32 lanes and the scale is a
// chain of several hundred cycles, so R of them run side by side.  row: -1 for none (warp-uniform).
template <int R>
__device__ __forceinline__ void quantise_rows(const Args& a, const int (&row)[R], int unit, int lane, int f, const float4 (&g)[R],
                                              const float4 (&u)[R]) {
    const int f0 = unit * QB + f;
    float h[R][4], am[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        h[i][0] = silu_mul(g[i].x, u[i].x);
        h[i][1] = silu_mul(g[i].y, u[i].y);
        h[i][2] = silu_mul(g[i].z, u[i].z);
        h[i][3] = silu_mul(g[i].w, u[i].w);
        am[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[i][e] = f0 + e < a.N ? h[i][e] : 0.f;
            am[i] = max_nan(am[i], fabsf(h[i][e]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < R; ++i) am[i] = max_nan(am[i], __shfl_xor_sync(0xFFFFFFFFu, am[i], o));
    }
    uint32_t v[R], held[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float is = inv_scale(group_scale(am[i], a.e8m0, held[i]));
        v[i] = pack4_e4m3(h[i][0] * is, h[i][1] * is, h[i][2] * is, h[i][3] * is);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (row[i] < 0) continue;
        uint8_t* dst = a.hq + (int64_t)row[i] * a.ld_hq + f0;
        if (f0 + 4 <= a.N) {
            *reinterpret_cast<uint32_t*>(dst) = v[i];
        } else {
            for (int e = 0; f0 + e < a.N; ++e) dst[e] = (uint8_t)(v[i] >> (8 * e));
        }
        if (lane == 0) {
            const int64_t at = (int64_t)unit * a.ld_hs + row[i];
            if (a.e8m0) static_cast<uint8_t*>(a.hs)[at] = (uint8_t)held[i];
            else static_cast<uint32_t*>(a.hs)[at] = held[i];
        }
    }
}

// Sum of 4 fp32 at `at` over the S CTAs, in rank order; all S loads are in flight at once.
template <int S>
__device__ __forceinline__ float4 sum_ranks(uint32_t at) {
    float4 v[S];
#pragma unroll
    for (int p = 0; p < S; ++p) v[p] = ld_cluster4(map_to_rank(at, p));
#pragma unroll
    for (int p = 1; p < S; ++p) v[0] = add4(v[0], v[p]);
    return v[0];
}

// Drain warp ew of CTA `rank` adds and finishes rows ew S + rank, + 8 S, ..., gated R at a time.  Loads from
// the peers run at about 15 bytes a cycle into an SM, which bounds this (128 x 256 sums: 4 to 5 us).
template <int BN, bool GATED, int S>
__device__ __forceinline__ void join_rows(const Args& a, uint32_t part0, int rank, int ew, int lane, int m0, int n0, int valid) {
    constexpr int R = GATED ? 8 / S : 1, STEP = EPI_WARPS * S;
#pragma unroll 1
    for (int r = ew * S + rank; r < valid; r += R * STEP) {
        uint32_t part[R];
        int row[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool in = r + i * STEP < valid;
            row[i] = in ? m0 + r + i * STEP : -1;
            part[i] = part0 + (uint32_t)((in ? r + i * STEP : r) * part_pitch(BN)) * 4u + 16u * lane;
        }
        if constexpr (GATED) {
            // Whole 512-byte runs of the row (a lane's own gate and up columns, 32 bytes of every 64, took
            // 1.4 times as long); each 16 columns are 8 gate, then 8 up, so lanes l and l ^ 2 swap halves.
            const bool up = (lane & 2) != 0;
            float4 g[R], u[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                g[i] = sum_ranks<S>(part[i]);
                u[i] = sum_ranks<S>(part[i] + 512);
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float4 give = up ? g[i] : u[i];
                const float4 got = make_float4(__shfl_xor_sync(0xFFFFFFFFu, give.x, 2), __shfl_xor_sync(0xFFFFFFFFu, give.y, 2),
                                               __shfl_xor_sync(0xFFFFFFFFu, give.z, 2), __shfl_xor_sync(0xFFFFFFFFu, give.w, 2));
                if (up) g[i] = got;
                else u[i] = got;
            }
            quantise_rows<R>(a, row, n0 / (2 * QB), lane, (lane >> 2) * 8 + (lane & 1) * 4 + (up ? 64 : 0), g, u);
        } else {
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 128) {
                const int c = c0 + 4 * lane;
                if (n0 + c >= a.N) break;
                float4 v[R];
#pragma unroll
                for (int i = 0; i < R; ++i) v[i] = sum_ranks<S>(part[i] + 4u * c0);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (row[i] < 0) continue;
                    const int64_t at = (int64_t)row[i] * a.ldy + n0 + c;
                    if (a.y_vec && n0 + c + 4 <= a.N) {
                        if (a.y_f32) {
                            *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = v[i];
                        } else {
                            __nv_bfloat162 lo = __floats2bfloat162_rn(v[i].x, v[i].y), hi = __floats2bfloat162_rn(v[i].z, v[i].w);
                            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) =
                                make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
                        }
                    } else {
                        const float e[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (n0 + c + j >= a.N) break;
                            if (a.y_f32) static_cast<float*>(a.y)[at + j] = e[j];
                            else static_cast<__nv_bfloat16*>(a.y)[at + j] = __float2bfloat16_rn(e[j]);
                        }
                    }
                }
            }
        }
    }
}
template <int BN, bool GATED>
__device__ __forceinline__ void join_partials(const Args& a, uint32_t part0, int rank, int ew, int lane, int m0, int n0, int valid) {
    if (a.S == 2) join_rows<BN, GATED, 2>(a, part0, rank, ew, lane, m0, n0, valid);
    else if (a.S == 4) join_rows<BN, GATED, 4>(a, part0, rank, ew, lane, m0, n0, valid);
    else join_rows<BN, GATED, 8>(a, part0, rank, ew, lane, m0, n0, valid);
}

// A block's scales as they were loaded: the token's (bits, or the e8m0 byte) and the weights'.
struct Fetched {
    uint32_t x;
    float w0, w1;
};

// GRP: K blocks per stage, per TMEM buffer and per commit.
template <int GRP, bool GATED>
__global__ void __launch_bounds__(NTHREADS, 1) fp8_gemm_kernel(const __grid_constant__ Maps maps, Args a) {
    constexpr int COLS = BUF_COLS / GRP;      // columns reserved per K block
    constexpr int HALF = COLS / 2;            // accumulators per thread
    constexpr int PIECE = 32;                 // columns per batch of tensor-memory loads (two batches in registers)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int w_bytes = a.bn * 128, a_bytes = a.a_rows * 128;
    const int stage_bytes = GRP * (w_bytes + a_bytes);
    uint8_t* tail = ring + a.stages * stage_bytes;
    float* amax_cta = reinterpret_cast<float*>(tail);                           // gated: [half][128]
    float* amax_all = amax_cta + 2 * BM;                                        // gated: [parity][rank][128], or staging
    __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[2], tempty[2], xbar[2], mma_done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a cluster shares a unit's K (S > 1), or the 128 features of a gated unit
    constexpr bool CAN_SPLIT = GRP == 1 || (GRP == 2 && !GATED);
    const bool shared_k = CAN_SPLIT && a.S > 1;
    const uint32_t crank = GATED || CAN_SPLIT ? cluster_rank() : 0u, cctas = GATED || CAN_SPLIT ? cluster_size() : 1u;
    const uint32_t rank = shared_k ? 0u : crank, csize = shared_k ? 1u : cctas;
    const int first = blockIdx.x / cctas, step = gridDim.x / cctas;   // units go to clusters
    const int groups = (a.kt + GRP - 1) / GRP, split = shared_k ? (int)crank : 0;
    const int g0 = groups * split / a.S, n_grp = groups * (split + 1) / a.S - g0;      // this CTA's groups of K blocks
    const int kb_end = min(a.kt, (g0 + n_grp) * GRP);

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], EPI_WARPS); mbar_init(&xbar[b], 1); }
        mbar_init(&mma_done, 1);
        fence_mbar_init();
        abort_flag = 0;
    }
    __syncthreads();
    if (GATED && csize > 1) cluster_arrive();   // waited for before anything is sent to a peer
    volatile int* abort = &abort_flag;

    // unit -> token tile and first weight row
    auto unit_rows = [&](int u, int& m0, int& n0) {
        const int mt = u / a.n_nt;
        m0 = mt * BM;
        n0 = ((u - mt * a.n_nt) * (int)csize + (int)rank) * a.bn;
    };

    if (warp < CTRL_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTRL_REGS));
        if (warp == 0) {
            // ------------------------------------------------ producer
            const uint32_t el = elect_one();
            if (el) {
                prefetch_map(&maps.w);
                prefetch_map(&maps.a);
            }
            const uint32_t ring0 = smem_addr(ring), full0 = smem_addr(full);
            auto copy_w = [&](int stage, int n0, int g) {
                const int kb = (g0 + g) * GRP;
                if (el) {
                    expect_tx(full0 + 8 * stage, (uint32_t)(GRP * w_bytes + tokens_bytes(a.k_full, a.kt, kb, GRP, a_bytes)));
                    tma_load_3d(ring0 + stage * stage_bytes, &maps.w, 0, n0, kb, full0 + 8 * stage);
                }
            };
            auto copy_a = [&](int stage, int m0, int g) {
                if (el)
                    copy_tokens(maps, a.k_full, a.kt, ring0 + stage * stage_bytes + GRP * w_bytes, (g0 + g) * GRP, GRP, m0, a_bytes,
                                full0 + 8 * stage);
            };
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            bool ok = true;
            // the weights do not depend on the preceding kernel: the first unit's stages are
            // requested before the wait for it
            int pre = 0;
            {
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
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[stage], phase ^ 1u, a.wait_limit, a.status, abort));
                        if (!ok) break;
                        copy_w(stage, n0, g);
                    }
                    copy_a(stage, m0, g);
                    issued = min(issued + 1, a.stages);
                    if (++stage == a.stages) { stage = 0; phase ^= 1u; }
                }
            }
            // every issued copy lands before the CTA exits: the last `issued` stages, newest first
            for (; issued > 0; --issued) {
                if (--stage < 0) { stage = a.stages - 1; phase ^= 1u; }
                mbar_wait_bounded(&full[stage], phase, LANDING_LIMIT_US, a.status, nullptr);
            }
        } else if (warp == 1) {
            tc::tmem_alloc(&tmem_slot, 512);
            tc::tc_fence_before();
            named_bar_sync(2, (1 + EPI_WARPS) * 32);            // the drain warps read the address
            tc::tc_fence_after();
            pdl_wait();                      // no bounded wait before it: limits count this kernel's time alone
            // ------------------------------------------------ MMA issuer
            const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_slot, 0);
            const uint32_t el = elect_one();
            const uint32_t idesc = idesc_for(a.bn);
            const uint32_t d0 = (uint32_t)tc::sw128_desc(smem_addr(ring));
            int stage = 0, buf = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true, issued = false;
            const int stop = a.plant && blockIdx.x == 0 ? n_grp - 1 : -1;
            for (int u = first; u < a.n_units && ok; u += step) {
                for (int g = 0; g < n_grp; ++g) {
                    ok = g != stop && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[stage], phase, a.wait_limit, a.status, abort) &&
                                                     mbar_wait_bounded(&tempty[buf], tphase ^ 1u, a.wait_limit, a.status, abort));
                    if (!ok) break;
                    tc::tc_fence_after();
                    const int nk = min(GRP, kb_end - (g0 + g) * GRP);
                    uint32_t wd = d0 + (uint32_t)((stage * stage_bytes) >> 4);
                    uint32_t ad = wd + (uint32_t)((GRP * w_bytes) >> 4);
                    uint32_t dt = tmem + (uint32_t)(buf * BUF_COLS);
                    for (int i = 0; i < nk; ++i) {
                        mma_block(dt, ad, wd, idesc, el);
                        wd += (uint32_t)(w_bytes >> 4);
                        ad += (uint32_t)(a_bytes >> 4);
                        dt += (uint32_t)COLS;
                    }
                    if (el) {
                        tc::mma_commit(&tfull[buf]);
                        tc::mma_commit(&empty[stage]);
                    }
                    __syncwarp();
                    issued = true;
                    if (++stage == a.stages) { stage = 0; phase ^= 1u; }
                    if (++buf == 2) { buf = 0; tphase ^= 1u; }
                }
            }
            if (!ok && issued) finish_mmas(&mma_done, el, a.status);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        // ---------------------------------------------------- drain warps
        const int ew = warp - CTRL_WARPS;
        const int quarter = warp & 3, half = ew >> 2;
        const int r = quarter * 32 + lane;                     // token row of the tile = TMEM lane
        named_bar_sync(2, (1 + EPI_WARPS) * 32);
        tc::tc_fence_after();
        const uint32_t tmem = tmem_slot + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * HALF);
        pdl_wait();
        if (GATED && csize > 1) cluster_wait();
        EpiCtx ctx = {ew, quarter, half, lane, rank, csize, staging<GRP == 1>(tail, GATED, ew), amax_cta, amax_all, xbar, 0, 0u, abort};
        int buf = 0;
        uint32_t tphase = 0;
        bool dead = false;
        // What bounds the kernel is this warp's way round a group, so nothing but tensor memory is
        // waited for.  The scales come straight from global memory into registers, two groups ahead (a
        // unit's first ones before the last unit's results are written), and the MMA warp hands the
        // stage back itself.
        const float *sw0, *sw1;
        int rl;
        auto fetch = [&](Fetched (&f)[GRP], int g) {
#pragma unroll
            for (int i = 0; i < GRP; ++i) {
                const int kb = min((g0 + g) * GRP + i, a.kt - 1);
                const int64_t at = (int64_t)kb * a.ld_sa + rl;
                f[i].x = a.e8m0 ? (uint32_t)static_cast<const uint8_t*>(a.sa)[at] : static_cast<const uint32_t*>(a.sa)[at];
                f[i].w0 = sw0[kb];
                if (GATED || GRP > 1) f[i].w1 = sw1[kb];
            }
        };
        Fetched f0[GRP], f1[GRP], f2[GRP];                     // of groups 2, 1 and 0 at a unit's start
        auto fetch_unit = [&](int u) {
            int m0, n0;
            unit_rows(u, m0, n0);
            rl = min(m0 + r, a.M - 1);
            // gated: gate and up of the unit's features; plain: the tile's two scale blocks, or with
            // 256 rows the one that this half lies in
            const int blk = min(GATED ? n0 / (2 * QB) : (GRP == 1 ? n0 + half * HALF : n0) / QB, a.nblk - 1);
            sw0 = a.sw + (size_t)blk * a.kt;
            sw1 = a.sw + (size_t)(GATED ? blk + a.nblk : min(blk + 1, a.nblk - 1)) * a.kt;
            fetch(f2, 0);
            fetch(f1, 1);
            fetch(f0, 2);
        };
        if (first < a.n_units) fetch_unit(first);
        for (int u = first; u < a.n_units; u += step) {
            int m0, n0;
            unit_rows(u, m0, n0);
            const int valid = min(BM, a.M - m0);
            const bool live = quarter * 32 < valid;            // warp-uniform: some lane has a token
            const int col0 = n0 + half * HALF;                 // first weight-image row of this thread's columns
            // plain: bit p is set where the 16-column piece p lies in the second scale block
            uint32_t hi_mask = 0;
            if (!GATED) {
#pragma unroll
                for (int p = 0; p < HALF / 16; ++p) hi_mask |= ((col0 + 16 * p) / QB != n0 / QB) ? 1u << p : 0u;
            }
            float acc[HALF];
#pragma unroll
            for (int c = 0; c < HALF; ++c) acc[c] = 0.f;
            uint32_t pa[PIECE], pb[PIECE];
            auto scales_of = [&](const Fetched (&f)[GRP], float (&d0)[GRP], float (&d1)[GRP]) {
#pragma unroll
                for (int i = 0; i < GRP; ++i) {
                    const float x = a.e8m0 ? e8m0_to_f32((uint8_t)f[i].x) : __uint_as_float(f[i].x);
                    d0[i] = x * f[i].w0;
                    d1[i] = GATED || GRP > 1 ? x * f[i].w1 : 0.f;
                }
            };
            auto arrived = [&](bool ready) {
                if (!__all_sync(0xFFFFFFFFu, ready))
                    dead = !__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&tfull[buf], tphase, a.wait_limit, a.status, abort));
            };
            auto release = [&]() {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[buf]);
                if (++buf == 2) { buf = 0; tphase ^= 1u; }
            };
            if (!live) {
                for (int g = 0; g < n_grp && !dead; ++g) {
                    arrived(false);
                    release();
                }
            } else if (!dead) {
                float c0[GRP], c1[GRP];                        // combined scales of the group being drained
                auto add = [&](int g, int b, const uint32_t (&raw)[PIECE]) {
                    constexpr int RUN = HALF < PIECE ? HALF : PIECE;
#pragma unroll
                    for (int t0 = 0; t0 < PIECE; t0 += RUN) {
                        const int i = (b * PIECE + t0) / HALF;                     // block of the group
                        if (GRP > 1 && (g0 + g) * GRP + i >= kb_end) break;        // the last group may be partial
#pragma unroll
                        for (int t = t0; t < t0 + RUN; t += 2) {
                            const int c = (b * PIECE + t) % HALF;
                            const float k = (GATED ? (c & 8) != 0 : GRP > 1 && ((hi_mask >> (c / 16)) & 1u) != 0) ? c1[i] : c0[i];
                            tc::fma2(acc[c], acc[c + 1], raw[t], raw[t + 1], k);
                        }
                    }
                };
                // group g, whose first batch is on its way into pa; f: the scales of g + 1
                auto drain = [&](int g, Fetched (&f)[GRP]) {
                    const uint32_t tb = tmem + buf * BUF_COLS;
                    tc::tmem_wait_ld();
                    ld_batch<HALF, COLS, PIECE>(tb, 1, pb);
                    add(g, 0, pa);
                    tc::tmem_wait_ld();
                    ld_batch<HALF, COLS, PIECE>(tb, 2, pa);
                    add(g, 1, pb);
                    tc::tmem_wait_ld();
                    ld_batch<HALF, COLS, PIECE>(tb, 3, pb);
                    // a look at the next group's barrier takes about 100 cycles: the products hide it
                    const bool ready = mbar_test(&tfull[buf ^ 1], tphase ^ (uint32_t)buf);
                    add(g, 2, pa);
                    tc::tmem_wait_ld();
                    release();
                    float d0[GRP], d1[GRP];                    // the next group's; unused after the last
                    if (g + 1 < n_grp) {
                        arrived(ready);
                        if (dead) return;
                        tc::tc_fence_after();
                        ld_batch<HALF, COLS, PIECE>(tmem + buf * BUF_COLS, 0, pa);
                        scales_of(f, d0, d1);
                        fetch(f, g + 3);
                    }
                    add(g, 3, pb);
#pragma unroll
                    for (int i = 0; i < GRP; ++i) { c0[i] = d0[i]; c1[i] = d1[i]; }
                };
                arrived(false);
                if (!dead) {
                    tc::tc_fence_after();
                    ld_batch<HALF, COLS, PIECE>(tmem + buf * BUF_COLS, 0, pa);
                    scales_of(f2, c0, c1);
                    for (int g = 0; g < n_grp; g += 2) {
                        drain(g, f1);
                        if (dead || g + 1 >= n_grp) break;
                        drain(g + 1, f0);
                        if (dead) break;
                    }
                }
            }

            if constexpr (CAN_SPLIT) {
                if (shared_k) {
                    if (live) leave_partial<HALF>(reinterpret_cast<float*>(ring), half, r, acc);
                    tell_peers(dead, abort, a.S, lane);
                    cluster_arrive_release();
                    cluster_wait();
                    if (!*abort) join_partials<COLS, GATED>(a, smem_addr(ring), split, ew, lane, m0, n0, valid);
                    continue;
                }
            }
            if (u + step < a.n_units) fetch_unit(u + step);
            if constexpr (GATED) epi_gated<HALF>(a, ctx, acc, m0, n0, valid, dead);
            else if (live && !dead) epi_plain<HALF, GRP == 1>(maps.y, a, ctx, acc, m0, n0, valid);
        }
        if (!GATED && GRP == 1 && lane == 0) tma_store_done();
    }
    if (warp < CTRL_WARPS) {
        if (shared_k) cluster_arrive_release();                // the drain warps' barrier before they join
        if (shared_k || (GATED && csize > 1)) cluster_wait();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 1) tc::tmem_dealloc(tmem_slot, 512);
    if (shared_k || (GATED && csize > 1)) {     // nobody leaves while a peer may still reach into it
        cluster_arrive_release();
        cluster_wait();
        if (GATED) let_land(abort);
    }
}

// ------------------------------------------------------------------ launch
// Clusters of c CTAs (one per SM) that run at once: a cluster stays inside a GPC, and the GPCs' SMs
// are no multiple of it (152 SMs: 76 clusters of 2, 36 of 4, 15 of 8).
inline int cluster_slots(int sms, int c) { return c <= 2 ? sms / c : c == 4 ? sms * 95 / 400 : sms * 80 / 800; }

// Microseconds of a call, up to a constant, fitted to sweeps on this GPU (29 shapes, 70 to 3000 tokens, both
// scale types, every tile height and K range: the choice is within 0.7 % of the fastest of them on average).
// `waves` tiles of kr K blocks one after the other in a CTA, each with `fixed` for its start and its
// results, against the bytes of memory_bytes; each covers part of the other.
inline double plan_us(double waves, double kr, double block_us, double fixed, double memory_bytes) {
    const double cta = waves * (kr * block_us + fixed), hbm = memory_bytes / 6.8e6;
    return std::sqrt(cta * cta + hbm * hbm);
}
// Weights, and results at a third of the reading rate: all CTAs write theirs at about the same time.
inline double memory_bytes(const GemmCall& c, bool gated) {
    const double n = c.lin->d.out_features, rows = gated ? 2.0 * ((c.lin->d.out_features + QB - 1) / QB * QB) : n;
    return rows * c.lin->kt * 128.0 + 2.9 * c.M * n * (gated ? 1 : c.y_f32 ? 4 : 2);
}
// Joining S K ranges: sums of the tile's rows through distributed shared memory.
inline double join_us(bool gated, int bn, int S, int M, double ctas) {
    if (S == 1) return 0.0;
    return bn / 128.0 * (gated ? 1.55 * std::min(M, BM) / BM : 0.157 + 0.178 * S) + (gated ? 0.0054 : 0.0084) * ctas;
}
// The copies of a K block's operands into one SM run at about 118 GB/s.
inline double copy_us(int bn, int a_rows) { return (bn + a_rows) * 128.0 / 118e3; }

struct Plan {
    int grp, bn, cluster, units, n_nt, S;
    double us;                // the estimate it was chosen by
};

// Tensor maps of one call.  Token codes: [K block][row][128 B] (the K blocks of a row lie side by
// side), 128-byte swizzle; a ragged last block through [1][row][K], so that the copy fills zeros past
// K.  Weight image: [K block][row][128 B], swizzled already.  Rows and blocks past the end are filled
// with zeros.  scale_rows, scale_blocks: the box of the token scales' map ([K block][row]), 0 for none.
inline bool encode_maps(const GemmCall& c, const Args& a, int grp, int scale_rows, int scale_blocks, Maps* m) {
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t K = c.lin->d.in_features, kt = a.kt, M = c.M, Q = QB;
    const cuuint32_t one[3] = {1, 1, 1}, q = QB;
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto none = CU_TENSOR_MAP_INTERLEAVE_NONE;
    const auto wide = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    const auto fill = CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE;
    uint8_t* codes = const_cast<uint8_t*>(c.aq);
    const cuuint64_t as[2] = {(cuuint64_t)c.ld_aq, Q};
    bool ok = true;
    if (a.k_full > 0) {
        const cuuint64_t ad[3] = {Q, M, (cuuint64_t)a.k_full};
        const cuuint32_t ab[3] = {q, (cuuint32_t)a.a_rows, (cuuint32_t)grp};
        ok = enc(&m->a, u8, 3, codes, ad, as, ab, one, none, CU_TENSOR_MAP_SWIZZLE_128B, wide, fill) == CUDA_SUCCESS;
    }
    if (ok && a.k_full < a.kt) {
        const cuuint64_t ad[3] = {K, M, 1};
        const cuuint32_t ab[3] = {q, (cuuint32_t)a.a_rows, 1};
        ok = enc(&m->a_last, u8, 3, codes, ad, as, ab, one, none, CU_TENSOR_MAP_SWIZZLE_128B, wide, fill) == CUDA_SUCCESS;
        if (a.k_full == 0) m->a = m->a_last;      // a valid descriptor to prefetch
    }
    const cuuint64_t wd[3] = {Q, (cuuint64_t)a.rows_pad, kt}, ws[2] = {Q, (cuuint64_t)a.rows_pad * Q};
    const cuuint32_t wb[3] = {q, (cuuint32_t)a.bn, (cuuint32_t)grp};
    ok = ok && enc(&m->w, u8, 3, c.lin->w, wd, ws, wb, one, none, CU_TENSOR_MAP_SWIZZLE_NONE, wide, fill) == CUDA_SUCCESS;
    if (scale_rows > 0) {
        const cuuint64_t sd[2] = {M, kt}, ss[1] = {(cuuint64_t)(a.ld_sa * (a.e8m0 ? 1 : 4))};
        const cuuint32_t sb[2] = {(cuuint32_t)scale_rows, (cuuint32_t)scale_blocks};
        ok = ok && enc(&m->s, a.e8m0 ? u8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(c.as), sd, ss, sb, one, none,
                       CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, fill) == CUDA_SUCCESS;
    }
    if (a.y_tma) {
        const cuuint64_t yd[2] = {(cuuint64_t)a.N, M}, ys[1] = {(cuuint64_t)c.ldy * (c.y_f32 ? 4 : 2)};
        const cuuint32_t yb[2] = {c.y_f32 ? 32u : 64u, 32};
        ok = ok && enc(&m->y, c.y_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.y, yd, ys, yb, one, none,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, fill) == CUDA_SUCCESS;
    }
    return ok;
}

template <int GRP, bool GATED>
cudaError_t launch(const GemmCall& c, const Plan& p, Args& a, cudaStream_t s) {
    a.bn = p.bn;
    a.n_nt = p.n_nt;
    a.n_units = p.units;
    a.S = p.S;
    a.y_tma = !GATED && GRP == 1 && p.S == 1 && c.ldy * (c.y_f32 ? 4 : 2) % 16 == 0 && reinterpret_cast<uintptr_t>(c.y) % 16 == 0;
    Maps maps;
    if (!encode_maps(c, a, GRP, 0, 0, &maps)) return cudaErrorInvalidValue;
    const int cost = stage_cost(GRP, a.bn, a.a_rows), fixed = 1024 + tail_bytes(GRP, GATED);
    const int groups = (a.kt + GRP - 1) / GRP;
    a.stages = std::max(1, std::min(MAX_STAGES, (SMEM_MAX - fixed) / cost));
    if (p.S == 1) a.stages = std::min(a.stages, std::max(2, groups));      // S > 1 also keeps its sums there
    const int smem = fixed + a.stages * cost;
    if (p.S > 1 && a.stages * GRP * (a.bn + a.a_rows) * 128 < BM * part_pitch(a.bn) * 4) return cudaErrorInvalidValue;
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
    if (p.cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = p.cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    int slots = c.lin->num_sms;
    if (p.S > 1) {
        slots = p.units;                      // one unit per cluster
    } else if (p.cluster > 1) {
        // clusters that fit at once (a cluster stays inside one GPC), asked once: every plan of
        // this kernel without K ranges has the same cluster size and one CTA per SM
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
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<GRP, GATED>, maps, a);
}

inline Args base_args(const GemmCall& c) {
    Args a = {};
    a.y = c.y; a.ldy = c.ldy; a.y_f32 = c.y_f32;
    // four columns per store are 16 bytes of fp32 or 8 of bf16; eight of bf16 are 16
    a.y_vec = c.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(c.y) % (c.y_f32 ? 16 : 8) == 0;
    a.y_wide = !c.y_f32 && c.ldy % 8 == 0 && reinterpret_cast<uintptr_t>(c.y) % 16 == 0;
    a.hq = c.hq; a.ld_hq = c.ld_hq; a.hs = c.hs; a.ld_hs = c.ld_hs;
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
    a.k_full = L->d.in_features / QB;
    a.status = L->dev_status;
    a.wait_limit = L->wait_limit;
    a.plant = c.plant;
    return a;
}

}  // namespace dg
}  // namespace moe
