// Products with 4-bit weights, many rows per matrix, on the 5th-generation
// tensor cores (tcgen05, sm_103a).
//
// A tile is 128 weight rows (the MMA's M, tensor-memory lanes) by up to BN
// rows of x (its N, columns), a stage 256 input channels in two halves.  Four
// warps widen the codes, less their zero points, to bf16, exactly, and store
// them straight into tensor memory as the MMA's first operand: through shared
// memory each weight would be written and read there at two bytes, as long as
// the MMAs of 64 columns take.  Four warps drain; of the rest one brings codes,
// scales and zero points (bulk copies), one the rows of x (TMA, gathered by
// token where there are tokens) and one issues the MMAs.  Rows of x off the
// 16-byte grid, which TMA does not take, are brought by ten warps.
//
// The tensor core's running sum truncates, and scales are per 32 channels at
// the finest: each half goes into fresh accumulators, CHUNKS of them (1, 2 or
// 4, of 128, 64 or 32 channels, as fine as the groups), which the drain warps
// scale and add up in fp32 registers.  A lane is one weight row, so a scale is
// one scalar per thread and chunk.  Tensor memory holds 128 columns of
// accumulators per half, so that BN = 128 / CHUNKS, and two stages of operands.
//
#include <algorithm>

#include "dense_internal.cuh"
#include "int4.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int DRAIN_WARPS = 4, WIDEN_WARPS = 4;
constexpr int CODE_WARP = DRAIN_WARPS + WIDEN_WARPS, MMA_WARP = CODE_WARP + 1, X_WARP = MMA_WARP + 1;

enum XMode { X_TILE, X_GATHER, X_COPY };

// Warps that bring x, and the register split of setmaxnreg: the drain warps rise to DRAIN_REGS, the others drop
// to OTHER_REGS, of LAUNCH_REGS per thread.  (A warpgroup is four warps: without the copying warps one idles.)
template <XMode MODE>
struct Shape {
    static constexpr int X_WARPS = MODE == X_COPY ? 10 : 1;
    static constexpr int THREADS = MODE == X_COPY ? 640 : 384;
    static constexpr int LAUNCH_REGS = MODE == X_COPY ? 96 : 168;
    static constexpr int DRAIN_REGS = MODE == X_COPY ? 208 : 232, OTHER_REGS = MODE == X_COPY ? 64 : 136;
    static_assert(X_WARP + X_WARPS <= THREADS / 32, "warps");
    static_assert(DRAIN_WARPS * 32 * DRAIN_REGS + (THREADS - DRAIN_WARPS * 32) * OTHER_REGS <= THREADS * LAUNCH_REGS, "register split");
};

constexpr int HALF_K = 128, HALF_TILES = 2;      // channels, 64-channel tiles
constexpr int STAGE_K = 256, STAGE_TILES = 4;
constexpr int STAGES = 2;                        // widened operands in tensor memory
constexpr int COLS = 128;                        // accumulator columns of a half
constexpr int A_COLS = STAGE_K / 2;              // operand columns of a stage: two bf16 channels each
constexpr int A_BASE = 2 * COLS;
static_assert(A_BASE + STAGES * A_COLS <= 512, "tensor memory");
constexpr int RING = 4;                          // codes: 16 KB a stage
// Scales are needed until a stage is drained.  Their slots need no barrier to become free: who hands back
// codes of stage n - RING has seen the MMAs of n - RING - STAGES complete, and those waited for the draining
// of the stage before.
constexpr int SCALE_RING = 8;
static_assert(SCALE_RING >= RING + STAGES + 1, "scales");
constexpr int X_RING = 8;                        // halves of x at most
constexpr int X_BOX = 32;                        // rows of x that one copy brings
constexpr int DONE = 8;                          // stages whose completion can be asked for

template <int CHUNKS>
struct Smem {
    static constexpr int BN = COLS / CHUNKS;
    uint8_t x[(CHUNKS == 4 ? 64 : 128) * 1024];  // halves of two tiles of bn rows, 128-byte swizzle, 1024-byte aligned
    uint4 codes[RING][STAGE_TILES][I4_STRIP][32];
    uint32_t zeros[RING][2 * CHUNKS][I4_STRIP][8];
    uint2 scales[SCALE_RING][2 * CHUNKS][I4_STRIP][8];   // per chunk fp32 pairs; bf16 pairs fill the first half of a stage's
    uint64_t code_full[RING], code_free[RING], scale_full[SCALE_RING];
    uint64_t a_full[STAGES], x_full[X_RING], done[2][DONE], drained[2], last;
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

// Tries a wait up to 256 times, in the fewest instructions: what waiting warps issue the others lack.
__device__ __forceinline__ bool try_wait_many(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 0;\n"
        "AGAIN:\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
        " @p bra OVER;\n add.u32 n, n, 1;\n setp.lt.u32 q, n, 256;\n @q bra AGAIN;\n"
        "OVER:\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}

// As mbar_wait_bounded.  PATIENT: by a warp that works ahead and can sleep between its looks.
template <bool PATIENT>
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, uint32_t limit_us, uint32_t* status, volatile int* abort) {
    if (PATIENT ? mbar_try_wait(bar, parity) : try_wait_many(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (true) {
        if (PATIENT) __nanosleep(100);
        if (PATIENT ? mbar_try_wait(bar, parity) : try_wait_many(bar, parity)) return true;
        if (*abort) return false;
        if (global_ns() - t0 > (uint64_t)limit_us * 1000ull) {
            atomicOr(status, MOE_DEV_WAIT_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
}

// (a0, a1) += (p0, p1) * (s, s): two fp32 fused multiply-adds in one instruction.
__device__ __forceinline__ void fma_pair(uint64_t& a, uint32_t p0, uint32_t p1, uint64_t ss) {
    asm("{\n .reg .b64 t;\n mov.b64 t, {%1, %2};\n fma.rn.f32x2 %0, t, %3, %0;\n}" : "+l"(a) : "r"(p0), "r"(p1), "l"(ss));
}

// D f32, A = B = bf16, both K-major, M = 128.
__device__ __forceinline__ uint32_t idesc_for(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

template <int CHUNKS, XMode MODE, bool ZEROS, bool GATED>
__global__ void __launch_bounds__(Shape<MODE>::THREADS, 1) int4_many_kernel(const __grid_constant__ CUtensorMap x_map, const Int4Call c, int bn,
                                                                               int x_slots) {
    using S = Smem<CHUNKS>;
    constexpr int NTHREADS = Shape<MODE>::THREADS, X_WARPS = Shape<MODE>::X_WARPS;
    constexpr int BN = S::BN;                    // columns reserved per chunk; bn, at most that, rows per tile
    constexpr int CHUNK_STEPS = 4 / CHUNKS;      // 32-channel steps of a chunk
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int* start = sm.table;
    int* first = sm.table + c.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int feature_tiles = c.strips;
    const int stages = (c.kt + STAGE_TILES - 1) / STAGE_TILES;      // per unit

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(&sm.a_full[s], WIDEN_WARPS);
        for (int s = 0; s < X_RING; ++s) mbar_init(&sm.x_full[s], X_WARPS);
        for (int s = 0; s < DONE; ++s) {
            mbar_init(&sm.done[0][s], 1);
            mbar_init(&sm.done[1][s], 1);
        }
        for (int s = 0; s < RING; ++s) {
            mbar_init(&sm.code_full[s], 1);
            mbar_init(&sm.code_free[s], WIDEN_WARPS);
        }
        for (int s = 0; s < SCALE_RING; ++s) mbar_init(&sm.scale_full[s], 1);
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
    i4::row_tiles<NTHREADS>(c, bn, start, first);
    constexpr uint32_t tmem = 0;                 // where an allocation of all 512 columns starts
    volatile int* abort = &sm.abort;
    const int units = start[c.E] * feature_tiles;
    auto unit_at = [&](int u) { return i4::unit_at(c, u, feature_tiles, bn, start, first); };
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, wait_bounded<false>(bar, parity, c.wait_limit, c.status, abort));
    };
    auto patient_wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, wait_bounded<true>(bar, parity, c.wait_limit, c.status, abort));
    };
    // waits until the MMAs of half h of stage n are complete
    auto done = [&](int h, uint32_t n) { return warp_wait(&sm.done[h][n % DONE], n / DONE & 1u); };

    if (warp >= DRAIN_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Shape<MODE>::OTHER_REGS));
        if (warp < CODE_WARP) {
            // ------------------------------------------------------------ codes into tensor memory
            pdl_wait();                          // no bounded wait before it: limits count this kernel's time alone
            const int w = warp - DRAIN_WARPS, g = lane >> 2;         // blocks 2 w and 2 w + 1
            const uint32_t to = tmem + ((uint32_t)(w * 32) << 16) + A_BASE;
            int at = 0;
            uint32_t code_phase = 0, n = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                for (int st = 0; st < stages; ++st, ++n) {
                    ok = warp_wait(&sm.code_full[at], code_phase);
                    if (!ok) break;
                    ok = n < STAGES || done(1, n - STAGES);
                    if (!ok) break;
                    const int slot = n % STAGES;
                    tc::tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int block = 2 * w + i;
#pragma unroll
                        for (int tile = 0; tile < STAGE_TILES; ++tile) {
                            uint32_t r[16], v[4];
                            if (STAGE_TILES * st + tile < c.kt) {
                                const uint4 code = sm.codes[at][tile][block][lane];
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    const uint32_t z = ZEROS ? sm.zeros[at][(tile * 2 + half) / CHUNK_STEPS][block][g] : I4_ZERO;
                                    i4::widen(half ? code.y : code.x, ZEROS ? __byte_perm(z, 0, 0x1010) : z, v);
                                    r[8 * half] = v[0], r[8 * half + 1] = v[1], r[8 * half + 4] = v[2], r[8 * half + 5] = v[3];
                                    i4::widen(half ? code.w : code.z, ZEROS ? __byte_perm(z, 0, 0x3232) : z, v);
                                    r[8 * half + 2] = v[0], r[8 * half + 3] = v[1], r[8 * half + 6] = v[2], r[8 * half + 7] = v[3];
                                }
                            } else {             // channels past the image
#pragma unroll
                                for (int e = 0; e < 16; ++e) r[e] = 0u;
                            }
                            tmem_st_16x32(to + ((uint32_t)(i * 16) << 16) + slot * A_COLS + tile * (A_COLS / STAGE_TILES), r);
                        }
                    }
                    tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.code_free[at]);
                        mbar_arrive(&sm.a_full[slot]);
                    }
                    if (++at == RING) { at = 0; code_phase ^= 1u; }
                }
            }
        } else if (warp == CODE_WARP) {
            // ------------------------------------------------------------ codes, scales, zero points
            const uint32_t el = elect_one();
            const int s_rec = (c.s_f32 ? 8 : 4) * I4_STRIP * 8, z_rec = 4 * I4_STRIP * 8;    // bytes of a strip's group
            uint32_t n = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const i4::Unit un = unit_at(u);
                const size_t strip = (size_t)un.expert * c.strips + un.tile;
                const char* w = reinterpret_cast<const char*>(c.w) + strip * c.kt * (I4_STRIP * 512);
                const char* s = c.s + strip * c.groups * s_rec;
                const char* z = reinterpret_cast<const char*>(c.z) + strip * c.groups * z_rec;
                for (int st = 0; st < stages; ++st, ++n) {
                    // the weights do not depend on the preceding kernel: the first of them are requested before the wait for it
                    if (n == RING) pdl_wait();
                    const uint32_t slot = n % RING, s_slot = n % SCALE_RING;
                    ok = n < RING || patient_wait(&sm.code_free[slot], (n / RING & 1u) ^ 1u);
                    if (!ok) break;
                    const int tiles = min(STAGE_TILES, c.kt - st * STAGE_TILES), bytes = tiles * (I4_STRIP * 512);
                    // a record for every chunk, whatever the groups: neighbours where groups are as long as chunks
                    const int step = st * (2 * STAGE_TILES), chunks = (2 * tiles + CHUNK_STEPS - 1) / CHUNK_STEPS;
                    const int pieces = c.groups_are_chunks ? 1 : chunks, records = c.groups_are_chunks ? chunks : 1;
                    if (el) {
                        mbar_arrive_expect_tx(&sm.code_full[slot], bytes + (ZEROS ? chunks * z_rec : 0));
                        bulk_g2s(sm.codes[slot], w + (size_t)st * (STAGE_TILES * I4_STRIP * 512), bytes, &sm.code_full[slot]);
                        mbar_arrive_expect_tx(&sm.scale_full[s_slot], chunks * s_rec);
#pragma unroll 1
                        for (int j = 0; j < pieces; ++j) {
                            const size_t from = i4::group_of(c, step + j * CHUNK_STEPS);
                            if (ZEROS)
                                bulk_g2s(reinterpret_cast<char*>(sm.zeros[slot]) + j * z_rec, z + from * z_rec, records * z_rec, &sm.code_full[slot]);
                            bulk_g2s(reinterpret_cast<char*>(sm.scales[s_slot]) + j * s_rec, s + from * s_rec, records * s_rec, &sm.scale_full[s_slot]);
                        }
                    }
                    __syncwarp();
                }
            }
            // every issued copy lands before the CTA exits
            for (uint32_t i = n - min(n, (uint32_t)SCALE_RING); i < n; ++i) {
                if (i + RING >= n) mbar_wait_bounded(&sm.code_full[i % RING], i / RING & 1u, LANDING_LIMIT_US, c.status, nullptr);
                mbar_wait_bounded(&sm.scale_full[i % SCALE_RING], i / SCALE_RING & 1u, LANDING_LIMIT_US, c.status, nullptr);
            }
        } else if (warp == MMA_WARP) {
            // ------------------------------------------------------------ MMA issuer
            pdl_wait();
            const uint32_t el = elect_one();
            const uint32_t b0 = (uint32_t)tc::sw128_desc(smem_addr(sm.x));
            const uint32_t tile_step = (uint32_t)(bn * 128) >> 4;
            uint32_t n = 0, xs = 0, x_phase = 0;
            bool ok = true, any = false;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const i4::Unit un = unit_at(u);
                const uint32_t idesc = idesc_for((un.count + 15) / 16 * 16);
                for (int st = 0; st < stages && ok; ++st, ++n) {
                    const uint32_t slot = n % STAGES;
                    ok = warp_wait(&sm.a_full[slot], n / STAGES & 1u);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && warp_wait(&sm.x_full[xs], x_phase) && warp_wait(&sm.drained[h], (n & 1u) ^ 1u);
                        if (!ok) break;
                        tc::tc_fence_after();
                        const uint32_t a = tmem + A_BASE + slot * A_COLS + h * (A_COLS / 2), d = tmem + h * COLS;
                        const uint32_t b = b0 + xs * (HALF_TILES * tile_step);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_ts2(d + i / CHUNK_STEPS * BN, a + i * 16, b + (i >> 1) * tile_step + (i & 1) * 4, idesc, el, i % CHUNK_STEPS != 0);
                        if (el) tc::mma_commit(&sm.done[h][n % DONE]);
                        __syncwarp();
                        any = true;
                        if (++xs == x_slots) { xs = 0; x_phase ^= 1u; }
                    }
                }
            }
            // every issued MMA must complete before the tensor memory is released
            if (any) {
                if (el) tc::mma_commit(&sm.last);
                __syncwarp();
                mbar_wait_bounded(&sm.last, 0u, LANDING_LIMIT_US, c.status, nullptr);
            }
        } else if (warp < X_WARP + X_WARPS) {
            // ------------------------------------------------------------ rows of x into shared memory
            pdl_wait();
            const int xw = warp - X_WARP;
            const uint32_t tile_bytes = bn * 128;
            uint32_t n = 0, xs = 0;              // halves
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const i4::Unit un = unit_at(u);
                int row[4];
                if (MODE == X_GATHER) {          // lane i has rows 4 i to 4 i + 3; -1 reads as zeros
#pragma unroll
                    for (int i = 0; i < 4; ++i) row[i] = lane * 4 + i < un.count ? i4::source_row(c, un.row0 + lane * 4 + i) : -1;
                }
                for (int st = 0; st < 2 * stages; ++st, ++n) {
                    const uint32_t before = n - x_slots;
                    ok = n < x_slots || patient_wait(&sm.done[before & 1][before / 2 % DONE], before / 2 / DONE & 1u);
                    if (!ok) break;
                    uint8_t* const slot = sm.x + xs * (HALF_TILES * tile_bytes);
                    const uint32_t bar = smem_addr(&sm.x_full[xs]), to = smem_addr(slot);
                    if (MODE == X_TILE) {
                        const int boxes = (un.count + X_BOX - 1) / X_BOX;
                        if (lane == 0) mbar_arrive_expect_tx(&sm.x_full[xs], boxes * (HALF_TILES * X_BOX * 128));
                        __syncwarp();
                        const int box = lane / HALF_TILES, tile = lane % HALF_TILES;
                        if (box < boxes)
                            tma_rows(to + tile * tile_bytes + box * (X_BOX * 128), &x_map, st * HALF_K + tile * I4_K, un.row0 + box * X_BOX, bar);
                    } else if (MODE == X_GATHER) {
                        const int fours = (un.count + 3) / 4;
                        if (lane == 0) mbar_arrive_expect_tx(&sm.x_full[xs], fours * (HALF_TILES * 512));
                        __syncwarp();
                        if (lane < fours) {
#pragma unroll
                            for (int tile = 0; tile < HALF_TILES; ++tile)
                                tma_gather(to + tile * tile_bytes + lane * 512, &x_map, st * HALF_K + tile * I4_K, row, bar);
                        }
                    } else {
                        // a warp's lanes take 8 rows by 4 of the 16 pieces of 8 channels
                        constexpr int BATCH = 4;
                        const int r8 = lane >> 2;
#pragma unroll 1
                        for (int r0 = xw * 8; r0 < un.count; r0 += X_WARPS * 8) {
                            const int r = r0 + r8;
                            const int from = r < un.count ? i4::source_row(c, un.row0 + r) : -1;
                            const uint16_t* p = c.x + (from < 0 ? 0 : from) * c.ldx + st * HALF_K;
                            uint4 v[BATCH];
#pragma unroll
                            for (int i = 0; i < BATCH; ++i) {
                                const int k = ((lane & 3) + 4 * i) * 8;
                                v[i] = i4::load8(p + k, from < 0 ? 0 : min(c.K - st * HALF_K - k, 8));
                            }
                            if (r < un.count) {
#pragma unroll
                                for (int i = 0; i < BATCH; ++i) {
                                    const int piece = (lane & 3) + 4 * i;
                                    *reinterpret_cast<uint4*>(slot + (piece >> 3) * tile_bytes + r * 128 + (((piece & 7) ^ (r & 7)) << 4)) = v[i];
                                }
                            }
                        }
                        fence_async_proxy();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.x_full[xs]);
                    }
                    if (++xs == x_slots) xs = 0;
                }
            }
            // every issued copy lands before the CTA exits
            if (MODE != X_COPY)
                for (uint32_t i = n - min(n, (uint32_t)x_slots); i < n; ++i)
                    mbar_wait_bounded(&sm.x_full[i % x_slots], i / x_slots & 1u, LANDING_LIMIT_US, c.status, nullptr);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- drain, scale, add up
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Shape<MODE>::DRAIN_REGS));
        constexpr int PIECES = BN / 32;                      // of 32 columns, per chunk; four per half
        const uint32_t from = tmem + ((uint32_t)(warp * 32) << 16);
        const int row = warp * 32 + lane, block = row >> 4, g = row & 7, upper = (row >> 3) & 1;
        // where the row's scale lies in a record, in words, and which of its bytes make it an fp32
        const int s_at = (block * 8 + g) * (c.s_f32 ? 2 : 1) + (c.s_f32 ? upper : 0), s_step = I4_STRIP * 8 * (c.s_f32 ? 2 : 1);
        const uint32_t s_bytes = c.s_f32 ? 0x3210u : upper ? 0x3244u : 0x1044u;
        pdl_wait();
        uint32_t n = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const i4::Unit un = unit_at(u);
            uint64_t acc[PIECES][16];
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[p][i] = 0;
            for (int st = 0; st < stages && ok; ++st, ++n) {
                const uint32_t at = n % SCALE_RING;
                ok = warp_wait(&sm.scale_full[at], n / SCALE_RING & 1u);
                const uint32_t* s = reinterpret_cast<const uint32_t*>(sm.scales[at]) + s_at;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint64_t sc[CHUNKS];
#pragma unroll
                    for (int j = 0; j < CHUNKS; ++j) {
                        uint32_t v = __byte_perm(s[(h * CHUNKS + j) * s_step], 0, s_bytes);
                        // chunks of the last stage may lie past the matrix
                        if (st * (2 * STAGE_TILES) + (h * CHUNKS + j) * CHUNK_STEPS >= 2 * c.kt) v = 0;
                        sc[j] = (uint64_t)v << 32 | v;
                    }
                    ok = ok && done(h, n);       // tcgen05.ld below is warp-collective
                    if (!ok) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int b = 0; b < 4; b += 2) {
                        uint32_t part[2][32];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int j = (b + i) / PIECES, p = (b + i) % PIECES;
                            if (p * 32 < un.count) tc::tmem_ld32u(from + h * COLS + j * BN + p * 32, part[i]);
                        }
                        tc::tmem_wait_ld();
                        if (b == 2) {
                            tc::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sm.drained[h]);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int j = (b + i) / PIECES, p = (b + i) % PIECES;
                            if (p * 32 < un.count) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) fma_pair(acc[p][e], part[i][2 * e], part[i][2 * e + 1], sc[j]);
                            }
                        }
                    }
                }
            }
            if (!ok) break;
            const int n0 = GATED ? (un.tile * I4_STRIP + block) * 8 + g : un.tile * 128 + row;
            const bool mine = n0 < c.N && !(GATED && upper);
            auto store = [&](auto* y) {
#pragma unroll
                for (int p = 0; p < PIECES; ++p) {
                    const int m0 = p * 32;
                    if (m0 >= un.count) break;
                    auto* at = y + (un.row0 + m0) * c.ldy + n0;
#pragma unroll
                    for (int i = 0; i < 32; ++i, at += c.ldy) {
                        float v = __uint_as_float((uint32_t)(acc[p][i / 2] >> (32 * (i & 1))));
                        if (GATED) v = i4::gate(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
                        if (mine && m0 + i < un.count) i4::put_y(at, v);
                    }
                }
            };
            if (c.y_f32) store(static_cast<float*>(c.y));
            else store(static_cast<__nv_bfloat16*>(c.y));
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

template <int CHUNKS, XMode MODE, bool ZEROS, bool GATED>
cudaError_t launch(const moe_int4* L, const Int4Call& c, const CUtensorMap& map, cudaStream_t s) {
    constexpr int fixed = sizeof(Smem<CHUNKS>) + 1024;
    constexpr int most = fixed + 2 * (MOE_DISPATCH_MAX_EXPERTS + 1) * (int)sizeof(int);
    static_assert(most <= 227 * 1024 - 1024, "shared memory");
    cudaError_t e = ensure_smem_limit<int4_many_kernel<CHUNKS, MODE, ZEROS, GATED>>(most);
    if (e != cudaSuccess) return e;
    const int64_t tiles = c.strips;
    // rows per tile, and as many halves of x as fit
    const int bn = Smem<CHUNKS>::BN;
    const int x_slots = std::min(X_RING, (int)sizeof(Smem<CHUNKS>::x) / (bn * 128 * HALF_TILES));
    const int64_t row_tiles = c.offsets ? std::min<int64_t>(c.rows, c.rows / bn + c.E) : ((int64_t)c.rows + bn - 1) / bn;
    const int64_t grid = std::min<int64_t>(tiles * row_tiles, L->num_sms);
    return launch_pdl(int4_many_kernel<CHUNKS, MODE, ZEROS, GATED>, dim3((unsigned)grid), dim3(Shape<MODE>::THREADS),
                      fixed + 2 * (c.E + 1) * (int)sizeof(int), s, map, c, bn, x_slots);
}

template <int CHUNKS, XMode MODE>
cudaError_t launch_types(const moe_int4* L, const Int4Call& c, const CUtensorMap& map, cudaStream_t s) {
    if (c.gated) return c.z ? launch<CHUNKS, MODE, true, true>(L, c, map, s) : launch<CHUNKS, MODE, false, true>(L, c, map, s);
    return c.z ? launch<CHUNKS, MODE, true, false>(L, c, map, s) : launch<CHUNKS, MODE, false, false>(L, c, map, s);
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
    const int chunk = group % 128 == 0 || L->groups == 1 ? 128 : group % 64 == 0 ? 64 : 32;
    Int4Call call = c;
    call.groups_are_chunks = group == chunk;
    return chunk == 128 ? launch_mode<1>(L, call, s) : chunk == 64 ? launch_mode<2>(L, call, s) : launch_mode<4>(L, call, s);
}

}  // namespace moe
