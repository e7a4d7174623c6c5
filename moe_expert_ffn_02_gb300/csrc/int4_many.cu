// Products with 4-bit weights, many rows per matrix, on the 5th-generation
// tensor cores (tcgen05, sm_103a).
//
// A tile is 128 weight rows (the MMA's M, tensor-memory lanes) by up to BN
// rows of x (its N, columns), a stage 128 input channels.  Eight warps widen
// the codes, less their zero points, to bf16, exactly, and store them straight
// into tensor memory as the MMA's first operand: through shared memory each
// weight would be written and read there at two bytes, 256 clocks of that
// memory for a stage of 64 columns whose MMAs take 256.  Eight warps drain;
// of the rest one brings codes, scales and zero points (bulk copies), one the
// rows of x (TMA, gathered by token where there are tokens) and one issues the
// MMAs.  Rows of x off the 16-byte grid, which TMA does not take, are brought
// by six warps.
//
// The tensor core's running sum truncates, and scales are per 32 channels at
// the finest: each stage goes into fresh accumulators, CHUNKS of them (1, 2 or
// 4, of 128, 64 or 32 channels, as fine as the groups), which the drain warps
// scale and add up in fp32 registers.  A lane is one weight row, so a scale is
// one scalar per thread and chunk.  Tensor memory holds two sets of 128 columns
// of accumulators, so that BN = 128 / CHUNKS, and four stages of operands.
#include <algorithm>

#include "dense_internal.cuh"
#include "int4.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int DRAIN_WARPS = 8, WIDEN_WARPS = 8, X_WARPS = 6;
constexpr int CODE_WARP = DRAIN_WARPS + WIDEN_WARPS, MMA_WARP = CODE_WARP + 1, X_WARP = MMA_WARP + 1;
constexpr int NTHREADS = (X_WARP + X_WARPS) * 32;        // 768: six warpgroups
// setmaxnreg: launched at 80 per thread (768 x 80 = 61,440); the drain warps rise to 120, the others drop
// to 56: 8 * 32 * 120 + 16 * 32 * 56 = 59,392
constexpr int DRAIN_REGS = 120, OTHER_REGS = 56;
static_assert(DRAIN_WARPS * 32 * DRAIN_REGS + (NTHREADS - DRAIN_WARPS * 32) * OTHER_REGS <= NTHREADS * 80, "register split");

constexpr int STAGE_K = 128, STAGE_TILES = 2;    // channels; 64-channel tiles
constexpr int STAGES = 4;                        // operands of the MMA
constexpr int RING = 6;                          // codes: 8 KB a stage, to keep some 40 KB in flight
constexpr int COLS = 128;                        // accumulator columns of one set, two sets
constexpr int A_COLS = STAGE_K / 2;              // operand columns of a stage: two bf16 channels each
constexpr int A_BASE = 2 * COLS;
static_assert(A_BASE + STAGES * A_COLS <= 512, "tensor memory");
constexpr int X_BOX = 32;                        // rows of x that one copy brings

// A stage of a strip as it is copied: its tiles and the records of the groups that it meets.
template <int CHUNKS>
struct Codes {
    uint4 w[STAGE_TILES][I4_STRIP][32];
    uint2 s[CHUNKS][I4_STRIP][8];                // fp32 pairs; bf16 pairs fill the first half
    uint32_t z[CHUNKS][I4_STRIP][8];
};

template <int CHUNKS>
struct Smem {
    static constexpr int BN = COLS / CHUNKS;
    uint8_t x[STAGES][STAGE_TILES][BN * 128];    // 128-byte swizzle, 1024-byte aligned
    Codes<CHUNKS> ring[RING];
    uint64_t full[STAGES], done[STAGES], drained[2], last;
    uint64_t code_full[RING], code_free[RING];
    uint32_t tmem;
    int abort;
    int table[1];                                // start[E + 1], first[E + 1]
};

// 16 lanes by 32 columns, four 8-column groups: registers 4 i .. 4 i + 3 of lane 4 g + q are columns
// 8 i + 2 q, + 1 of row g, then of row g + 8.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two K16 steps (32 channels), the first operand in tensor memory, by the elected lane.  b_lo: low word of
// the second operand's descriptor, 2 more per step.  accumulate: whether the first adds to what is there.
__device__ __forceinline__ void mma_ts2(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t elected, uint32_t accumulate) {
    constexpr uint32_t HI = (uint32_t)(tc::DESC_HI >> 32);
    asm volatile(
        "{\n .reg .pred q, t;\n .reg .b64 b;\n .reg .b32 x, y;\n"
        " setp.ne.b32 q, %5, 0;\n setp.ne.b32 t, %6, 0;\n"
        " mov.b64 b, {%2, %4};\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, t;\n"
        " setp.eq.b32 t, 0, 0;\n"
        " add.u32 x, %1, 8;\n add.u32 y, %2, 2;\n mov.b64 b, {y, %4};\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(idesc), "n"(HI), "r"(elected), "r"(accumulate)
        : "memory");
}

// True in one lane of a converged warp; the loops around it stay warp-uniform.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p;
}

__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int k, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(row), "r"(bar)
        : "memory");
}
// Four rows anywhere, one after the other at dst.
__device__ __forceinline__ void tma_gather(uint32_t dst, const CUtensorMap* map, int k, const int (&row)[4], uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar)
        : "memory");
}

// D f32, A = B = bf16, both K-major, M = 128.
__device__ __forceinline__ uint32_t idesc_for(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

enum XMode { X_TILE, X_GATHER, X_COPY };

template <int CHUNKS, XMode MODE, bool ZEROS>
__global__ void __launch_bounds__(NTHREADS, 1) int4_many_kernel(const __grid_constant__ CUtensorMap x_map, const Int4Call c) {
    using S = Smem<CHUNKS>;
    constexpr int BN = S::BN;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int* start = sm.table;
    int* first = sm.table + c.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int feature_tiles = c.strips;
    const int stages = (c.kt + STAGE_TILES - 1) / STAGE_TILES;      // per unit

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm.full[s], WIDEN_WARPS + (MODE == X_COPY ? X_WARPS : 1));
            mbar_init(&sm.done[s], 1);
        }
        for (int s = 0; s < RING; ++s) {
            mbar_init(&sm.code_full[s], 1);
            mbar_init(&sm.code_free[s], WIDEN_WARPS + DRAIN_WARPS);
        }
        for (int b = 0; b < 2; ++b) mbar_init(&sm.drained[b], DRAIN_WARPS);
        mbar_init(&sm.last, 1);
        fence_mbar_init();
        sm.abort = 0;
    }
    if (warp == 0) tc::tmem_alloc(&sm.tmem, 512);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (c.offsets) pdl_wait();
    i4::row_tiles<NTHREADS>(c, BN, start, first);
    const uint32_t tmem = sm.tmem;
    volatile int* abort = &sm.abort;
    const int units = start[c.E] * feature_tiles;
    auto unit_at = [&](int u) { return i4::unit_at(c, u, feature_tiles, BN, start, first); };
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, c.wait_limit, c.status, abort); };
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)); };

    if (warp >= DRAIN_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp < CODE_WARP) {
            // ------------------------------------------------------------ codes into tensor memory
            pdl_wait();                          // no bounded wait before it: limits count this kernel's time alone
            const int w = warp - DRAIN_WARPS, quarter = w & 3, block = quarter * 2 + (w >> 2), g = lane >> 2;
            const uint32_t to = tmem + ((uint32_t)(quarter * 32 + (w >> 2) * 16) << 16) + A_BASE;
            int slot = 0, at = 0;
            uint32_t phase = 0, code_phase = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                for (int st = 0; st < stages; ++st) {
                    ok = warp_wait(&sm.code_full[at], code_phase);
                    if (!ok) break;
                    const Codes<CHUNKS>& in = sm.ring[at];
                    uint4 code[STAGE_TILES];
                    uint32_t zero[4];
#pragma unroll
                    for (int tile = 0; tile < STAGE_TILES; ++tile) code[tile] = in.w[tile][block][lane];
                    if (ZEROS) {
                        const int g0 = i4::group_of(c, st * 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            zero[i] = in.z[CHUNKS == 1 ? 0 : min(i4::group_of(c, st * 4 + i) - g0, CHUNKS - 1)][block][g];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.code_free[at]);
                    if (++at == RING) { at = 0; code_phase ^= 1u; }
                    ok = warp_wait(&sm.done[slot], phase ^ 1u);
                    if (!ok) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int tile = 0; tile < STAGE_TILES; ++tile) {
                        uint32_t r[16], v[4];
                        if (STAGE_TILES * st + tile < c.kt) {
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const uint32_t z = ZEROS ? zero[tile * 2 + half] : I4_ZERO;
                                i4::widen(half ? code[tile].y : code[tile].x, ZEROS ? __byte_perm(z, 0, 0x1010) : z, v);
                                r[8 * half] = v[0], r[8 * half + 1] = v[1], r[8 * half + 4] = v[2], r[8 * half + 5] = v[3];
                                i4::widen(half ? code[tile].w : code[tile].z, ZEROS ? __byte_perm(z, 0, 0x3232) : z, v);
                                r[8 * half + 2] = v[0], r[8 * half + 3] = v[1], r[8 * half + 6] = v[2], r[8 * half + 7] = v[3];
                            }
                        } else {                 // channels past the image
#pragma unroll
                            for (int i = 0; i < 16; ++i) r[i] = 0u;
                        }
                        tmem_st_16x32(to + slot * A_COLS + tile * (A_COLS / STAGE_TILES), r);
                    }
                    tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.full[slot]);
                    if (++slot == STAGES) { slot = 0; phase ^= 1u; }
                }
            }
        } else if (warp == CODE_WARP) {
            // ------------------------------------------------------------ codes, scales, zero points
            const uint32_t el = elect_one();
            const int s_rec = (c.s_f32 ? 8 : 4) * I4_STRIP * 8, z_rec = 4 * I4_STRIP * 8;    // bytes of a strip's group
            int slot = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const i4::Unit un = unit_at(u);
                const size_t strip = (size_t)un.expert * c.strips + un.tile;
                const char* w = reinterpret_cast<const char*>(c.w) + strip * c.kt * (I4_STRIP * 512);
                const char* s = c.s + strip * c.groups * s_rec;
                const char* z = reinterpret_cast<const char*>(c.z) + strip * c.groups * z_rec;
                for (int st = 0; st < stages; ++st) {
                    if (issued == RING) pdl_wait();
                    ok = issued < RING || warp_wait(&sm.code_free[slot], phase ^ 1u);
                    if (!ok) break;
                    Codes<CHUNKS>& in = sm.ring[slot];
                    const int bytes = min(STAGE_TILES, c.kt - st * STAGE_TILES) * (I4_STRIP * 512);
                    const int g0 = i4::group_of(c, st * 4), groups = i4::group_of(c, min(st * 4 + 3, 2 * c.kt - 1)) - g0 + 1;
                    if (el) {
                        mbar_arrive_expect_tx(&sm.code_full[slot], bytes + groups * (s_rec + (ZEROS ? z_rec : 0)));
                        bulk_g2s(in.w, w + (size_t)st * (STAGE_TILES * I4_STRIP * 512), bytes, &sm.code_full[slot]);
                        bulk_g2s(in.s, s + (size_t)g0 * s_rec, groups * s_rec, &sm.code_full[slot]);
                        if (ZEROS) bulk_g2s(in.z, z + (size_t)g0 * z_rec, groups * z_rec, &sm.code_full[slot]);
                    }
                    __syncwarp();
                    issued = min(issued, RING) + 1;
                    if (++slot == RING) { slot = 0; phase ^= 1u; }
                }
            }
            // every issued copy lands before the CTA exits: the last ones, newest first
            for (issued = min(issued, RING); issued > 0; --issued) {
                if (--slot < 0) { slot = RING - 1; phase ^= 1u; }
                mbar_wait_bounded(&sm.code_full[slot], phase, LANDING_LIMIT_US, c.status, nullptr);
            }
        } else if (warp == MMA_WARP) {
            // ------------------------------------------------------------ MMA issuer
            pdl_wait();
            const uint32_t el = elect_one();
            const uint32_t b0 = (uint32_t)tc::sw128_desc(smem_addr(sm.x[0][0]));
            int slot = 0;
            uint32_t phase = 0, n = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const i4::Unit un = unit_at(u);
                const uint32_t idesc = idesc_for((un.count + 15) / 16 * 16);
                for (int st = 0; st < stages; ++st, ++n) {
                    ok = __all_sync(0xFFFFFFFFu, wait(&sm.drained[n & 1], ((n >> 1) & 1u) ^ 1u) && wait(&sm.full[slot], phase));
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint32_t a = tmem + A_BASE + slot * A_COLS, d = tmem + (n & 1) * COLS;
                    const uint32_t b = b0 + ((slot * (STAGE_TILES * BN * 128)) >> 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_ts2(d + i / (4 / CHUNKS) * BN, a + i * 16, b + (i >> 1) * ((BN * 128) >> 4) + (i & 1) * 4, idesc, el,
                                i % (4 / CHUNKS) != 0);
                    if (el) tc::mma_commit(&sm.done[slot]);
                    __syncwarp();
                    if (++slot == STAGES) { slot = 0; phase ^= 1u; }
                }
            }
            // every issued MMA must complete before the tensor memory is released
            if (n) {
                if (el) tc::mma_commit(&sm.last);
                __syncwarp();
                mbar_wait_bounded(&sm.last, 0u, LANDING_LIMIT_US, c.status, nullptr);
            }
        } else if (MODE == X_COPY || warp == X_WARP) {
            // ------------------------------------------------------------ rows of x into shared memory
            pdl_wait();
            const int xw = warp - X_WARP;
            int slot = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const i4::Unit un = unit_at(u);
                int row[4];
                if (MODE == X_GATHER) {          // lane i has rows 4 i to 4 i + 3; -1 reads as zeros
#pragma unroll
                    for (int i = 0; i < 4; ++i) row[i] = lane * 4 + i < un.count ? i4::source_row(c, un.row0 + lane * 4 + i) : -1;
                }
                for (int st = 0; st < stages; ++st) {
                    ok = warp_wait(&sm.done[slot], phase ^ 1u);
                    if (!ok) break;
                    const uint32_t bar = smem_addr(&sm.full[slot]), to = smem_addr(sm.x[slot][0]);
                    if (MODE == X_TILE) {
                        const int boxes = (un.count + X_BOX - 1) / X_BOX;
                        if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], boxes * (STAGE_TILES * X_BOX * 128));
                        __syncwarp();
                        const int box = lane >> 1, tile = lane & 1;
                        if (box < boxes)
                            tma_rows(to + tile * (BN * 128) + box * (X_BOX * 128), &x_map, st * STAGE_K + tile * I4_K, un.row0 + box * X_BOX, bar);
                    } else if (MODE == X_GATHER) {
                        const int fours = (un.count + 3) / 4;
                        if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], fours * (STAGE_TILES * 512));
                        __syncwarp();
                        if (lane < fours) {
#pragma unroll
                            for (int tile = 0; tile < STAGE_TILES; ++tile)
                                tma_gather(to + tile * (BN * 128) + lane * 512, &x_map, st * STAGE_K + tile * I4_K, row, bar);
                        }
                    } else {
                        // a warp's lanes take 8 rows by 4 of the 16 pieces of 8 channels
                        constexpr int BATCH = 4;
                        const int r8 = lane >> 2;
#pragma unroll 1
                        for (int r0 = xw * 8; r0 < un.count; r0 += X_WARPS * 8) {
                            const int r = r0 + r8;
                            const int from = r < un.count ? i4::source_row(c, un.row0 + r) : -1;
                            const uint16_t* p = c.x + (from < 0 ? 0 : from) * c.ldx + st * STAGE_K;
                            uint4 v[BATCH];
#pragma unroll
                            for (int i = 0; i < BATCH; ++i) {
                                const int k = ((lane & 3) + 4 * i) * 8;
                                v[i] = i4::load8(p + k, from < 0 ? 0 : min(c.K - st * STAGE_K - k, 8));
                            }
                            if (r < un.count) {
#pragma unroll
                                for (int i = 0; i < BATCH; ++i) {
                                    const int piece = (lane & 3) + 4 * i;
                                    *reinterpret_cast<uint4*>(sm.x[slot][piece >> 3] + r * 128 + (((piece & 7) ^ (r & 7)) << 4)) = v[i];
                                }
                            }
                        }
                        fence_async_proxy();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.full[slot]);
                    }
                    issued = min(issued + 1, STAGES);
                    if (++slot == STAGES) { slot = 0; phase ^= 1u; }
                }
            }
            // Every issued copy lands before the CTA exits.  (A stage that lacks other arrivals, after an expired wait, only
            // gives them their time.)
            if (MODE != X_COPY) {
                for (; issued > 0; --issued) {
                    if (--slot < 0) { slot = STAGES - 1; phase ^= 1u; }
                    mbar_wait_bounded(&sm.full[slot], phase, LANDING_LIMIT_US, c.status, nullptr);
                }
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- drain, scale, add up
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(DRAIN_REGS));
        constexpr int W = BN >= 64 ? 32 : 16, PIECES = BN / 2 / W;      // columns a load; loads per thread and chunk
        const int quarter = warp & 3, side = warp >> 2;
        const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + side * W;
        const int row = quarter * 32 + lane, block = row >> 4, g = row & 7, upper = (row >> 3) & 1;
        pdl_wait();
        int slot = 0, at = 0;
        uint32_t phase = 0, code_phase = 0, n = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const i4::Unit un = unit_at(u);
            float acc[PIECES][W];
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
#pragma unroll
                for (int i = 0; i < W; ++i) acc[p][i] = 0.f;
            for (int st = 0; st < stages; ++st, ++n) {
                ok = warp_wait(&sm.code_full[at], code_phase);
                if (!ok) break;
                float sc[CHUNKS];
                const int g0 = i4::group_of(c, st * 4);
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) {
                    const int rec = CHUNKS == 1 ? 0 : min(i4::group_of(c, st * 4 + j * (4 / CHUNKS)) - g0, CHUNKS - 1);
                    const uint32_t* s = reinterpret_cast<const uint32_t*>(sm.ring[at].s);
                    const int pair = (rec * I4_STRIP + block) * 8 + g;
                    const uint32_t v = c.s_f32 ? s[pair * 2 + upper] : s[pair];
                    sc[j] = __uint_as_float(c.s_f32 ? v : upper ? v & 0xFFFF0000u : v << 16);
                    // the last stage's second tile may lie past the matrix
                    if (CHUNKS > 1 && st * 4 + j * (4 / CHUNKS) >= 2 * c.kt) sc[j] = 0.f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.code_free[at]);
                if (++at == RING) { at = 0; code_phase ^= 1u; }
                ok = warp_wait(&sm.done[slot], phase);           // tcgen05.ld below is warp-collective
                if (!ok) break;
                if (++slot == STAGES) { slot = 0; phase ^= 1u; }
                tc::tc_fence_after();
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
                    for (int p = 0; p < PIECES; ++p)
                        if ((2 * p + side) * W < un.count) {
                            uint32_t part[W];
                            const uint32_t t = from + (n & 1) * COLS + j * BN + 2 * p * W;
                            if constexpr (W == 32) tc::tmem_ld32u(t, part);
                            else tc::tmem_ld16u(t, part);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < W; i += 2) tc::fma2(acc[p][i], acc[p][i + 1], part[i], part[i + 1], sc[j]);
                        }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.drained[n & 1]);
            }
            if (!ok) break;
            const int n0 = c.gated ? (un.tile * I4_STRIP + block) * 8 + g : un.tile * 128 + row;
            const bool mine = n0 < c.N && !(c.gated && upper);
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const int m = (2 * p + side) * W + i;
                    float v = acc[p][i];
                    if (c.gated) v = i4::gate(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
                    if (mine && m < un.count) i4::store_y(c, un.row0 + m, n0, v);
                }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

template <int CHUNKS, XMode MODE, bool ZEROS>
cudaError_t launch(const moe_int4* L, const Int4Call& c, const CUtensorMap& map, cudaStream_t s) {
    constexpr int fixed = sizeof(Smem<CHUNKS>) + 1024;
    constexpr int most = fixed + 2 * (MOE_DISPATCH_MAX_EXPERTS + 1) * (int)sizeof(int);
    static_assert(most <= 227 * 1024 - 1024, "shared memory");
    constexpr int bn = Smem<CHUNKS>::BN;
    cudaError_t e = ensure_smem_limit<int4_many_kernel<CHUNKS, MODE, ZEROS>>(most);
    if (e != cudaSuccess) return e;
    const int64_t tiles = c.strips;
    const int64_t row_tiles = c.offsets ? std::min<int64_t>(c.rows, c.rows / bn + c.E) : (c.rows + bn - 1) / bn;
    const int64_t grid = std::min<int64_t>(tiles * row_tiles, L->num_sms);
    return launch_pdl(int4_many_kernel<CHUNKS, MODE, ZEROS>, dim3((unsigned)grid), dim3(NTHREADS),
                      fixed + 2 * (c.E + 1) * (int)sizeof(int), s, map, c);
}

template <int CHUNKS, XMode MODE>
cudaError_t launch_types(const moe_int4* L, const Int4Call& c, const CUtensorMap& map, cudaStream_t s) {
    return c.z ? launch<CHUNKS, MODE, true>(L, c, map, s) : launch<CHUNKS, MODE, false>(L, c, map, s);
}

template <int CHUNKS>
cudaError_t launch_mode(const moe_int4* L, const Int4Call& c, cudaStream_t s) {
    CUtensorMap map = {};
    if (c.x_grid < 16) return launch_types<CHUNKS, X_COPY>(L, c, map, s);
    const EncodeTiledFn encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)c.K, (cuuint64_t)c.x_rows}, strides[1] = {(cuuint64_t)c.ldx * 2};
    const cuuint32_t box[2] = {I4_K, c.token ? 1u : (cuuint32_t)X_BOX}, step[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(c.x), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return c.token ? launch_types<CHUNKS, X_GATHER>(L, c, map, s) : launch_types<CHUNKS, X_TILE>(L, c, map, s);
}

}  // namespace

bool int4_takes_many(const Int4Call& c) { return (c.offsets ? c.rows / c.E : c.rows) > 32; }

cudaError_t launch_int4_many(const moe_int4* L, const Int4Call& c, cudaStream_t s) {
    const int group = L->d.group;
    if (group % 128 == 0 || L->groups == 1) return launch_mode<1>(L, c, s);
    return group % 64 == 0 ? launch_mode<2>(L, c, s) : launch_mode<4>(L, c, s);
}

}  // namespace moe
