// Products with 4-bit weights, many rows per matrix, on the 5th-generation
// tensor cores (tcgen05, sm_103a).
//
// A tile is 128 weight rows (the MMA's M, tensor-memory lanes) by up to BN
// rows of x (its N, columns), a stage 128 input channels.  Eight warps widen
// the codes, less their zero points, to bf16, exactly, and store them straight
// into tensor memory as the MMA's first operand: through shared memory each
// weight would be written and read there at two bytes, 256 clocks of that
// memory for a stage of 64 columns whose MMAs take 256.  Three warps bring x
// into swizzled shared memory, one issues the MMAs, eight drain.
//
// The tensor core's running sum truncates, and scales are per 32 channels at
// the finest: each stage goes into fresh accumulators, CHUNKS of them (1, 2 or
// 4, of 128, 64 or 32 channels, as fine as the groups), which the drain warps
// scale and add up in fp32 registers.  A lane is one weight row, so a scale is
// one scalar per thread and chunk.  Tensor memory holds two sets of 128 columns
// of accumulators, so that BN = 128 / CHUNKS, and four stages of operands.
#include <algorithm>

#include "int4.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int DRAIN_WARPS = 8, WIDEN_WARPS = 8, LOAD_WARPS = 3;
constexpr int NTHREADS = (DRAIN_WARPS + WIDEN_WARPS + LOAD_WARPS + 1) * 32;      // 640: five warpgroups
// setmaxnreg: launched at 96 per thread (640 x 96 = 61,440); the drain warps rise to 112, the others drop
// to 80: 8 * 32 * 112 + 12 * 32 * 80 = 59,392
constexpr int DRAIN_REGS = 112, OTHER_REGS = 80;
static_assert(DRAIN_WARPS * 32 * DRAIN_REGS + (NTHREADS - DRAIN_WARPS * 32) * OTHER_REGS <= NTHREADS * 96, "register split");

constexpr int BM_BLOCKS = 8;                     // 128 weight rows
constexpr int STAGE_K = 128, STAGE_TILES = 2;    // channels; 64-channel tiles
constexpr int STAGES = 4;
constexpr int COLS = 128;                        // accumulator columns of one set, two sets
constexpr int A_COLS = STAGE_K / 2;              // operand columns of a stage: two bf16 channels each
constexpr int A_BASE = 2 * COLS;
static_assert(A_BASE + STAGES * A_COLS <= 512, "tensor memory");
constexpr int CODE_DEPTH = 5;                    // stages of codes in flight per widening warp
constexpr int SCALE_DEPTH = 4;                   // stages of scales in flight per drain thread
constexpr uint32_t LANDING_LIMIT = 2000000u;      // us, of the wait for MMAs in flight, whatever the limit of the others
constexpr int LOAD_LAG = 2;                      // stages of x in flight behind the one being issued

template <int CHUNKS>
struct Smem {
    static constexpr int BN = COLS / CHUNKS;
    uint8_t x[STAGES][STAGE_TILES][BN * 128];    // 128-byte swizzle, 1024-byte aligned
    uint4 codes[WIDEN_WARPS][CODE_DEPTH][STAGE_TILES][32];
    uint32_t zeros[WIDEN_WARPS][CODE_DEPTH][STAGE_TILES * 2][8];
    uint32_t scales[SCALE_DEPTH][CHUNKS][DRAIN_WARPS * 32];
    uint64_t full[STAGES], done[STAGES], drained[2], last;
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

// kind::f16 with the first operand in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// D f32, A = B = bf16, both K-major, M = 128.
__device__ __forceinline__ uint32_t idesc_for(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

template <int CHUNKS>
__global__ void __launch_bounds__(NTHREADS, 1) int4_many_kernel(const Int4Call c, int bn) {
    using S = Smem<CHUNKS>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int* start = sm.table;
    int* first = sm.table + c.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int feature_tiles = (c.blocks + BM_BLOCKS - 1) / BM_BLOCKS;
    const int stages = (c.kt + STAGE_TILES - 1) / STAGE_TILES;      // per unit

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm.full[s], WIDEN_WARPS + LOAD_WARPS);
            mbar_init(&sm.done[s], 1);
        }
        for (int b = 0; b < 2; ++b) mbar_init(&sm.drained[b], DRAIN_WARPS);
        mbar_init(&sm.last, 1);
        fence_mbar_init();
        sm.abort = 0;
    }
    if (warp == 0) tc::tmem_alloc(&sm.tmem, 512);
    pdl_wait();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    i4::row_tiles<NTHREADS>(c, bn, start, first);
    const uint32_t tmem = sm.tmem;
    volatile int* abort = &sm.abort;
    const int units = start[c.E] * feature_tiles;
    auto unit_at = [&](int u) { return i4::unit_at(c, u, feature_tiles, bn, start, first); };
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, c.wait_limit, c.status, abort); };

    if (warp >= DRAIN_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp < DRAIN_WARPS + WIDEN_WARPS) {
            // ------------------------------------------------------------ codes into tensor memory
            const int w = warp - DRAIN_WARPS, quarter = w & 3, block = quarter * 2 + (w >> 2), g = lane >> 2;
            const uint32_t to = tmem + ((uint32_t)(quarter * 32 + (w >> 2) * 16) << 16) + A_BASE;
            int p_unit = blockIdx.x, p_stage = 0, p_slot = 0;
            const uint4* p_w = nullptr;
            size_t p_rec = 0;
            bool p_have = false;
            auto enter = [&](int u) {
                const i4::Unit un = unit_at(u);
                const int b = un.tile * BM_BLOCKS + block;
                const size_t at = (size_t)un.expert * c.blocks + b;
                p_have = b < c.blocks;
                p_w = c.w + at * c.kt * 32 + lane;
                p_rec = at * c.groups * 8 + (lane & 7);
            };
            auto copy_next = [&]() {
                if (p_unit < units) {
                    if (p_have) {
                        const int t = p_stage * STAGE_TILES;
                        i4::copy16(smem_addr(&sm.codes[w][p_slot][0][lane]), p_w);
                        if (t + 1 < c.kt) i4::copy16(smem_addr(&sm.codes[w][p_slot][1][lane]), p_w + 32);
                        if (c.z && 2 * t + (lane >> 3) < 2 * c.kt)
                            i4::copy_small<4>(smem_addr(&sm.zeros[w][p_slot][lane >> 3][lane & 7]),
                                              c.z + p_rec + (size_t)i4::group_of(c, 2 * t + (lane >> 3)) * 8);
                    }
                    p_w += STAGE_TILES * 32;
                    if (++p_stage == stages) {
                        p_stage = 0;
                        p_unit += gridDim.x;
                        if (p_unit < units) enter(p_unit);
                    }
                }
                p_slot = p_slot + 1 == CODE_DEPTH ? 0 : p_slot + 1;
                i4::copy_commit();
            };
            if (p_unit < units) enter(p_unit);
#pragma unroll 1
            for (int i = 0; i < CODE_DEPTH - 1; ++i) copy_next();
            uint32_t n = 0;
            int at = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                for (int st = 0; st < stages; ++st, ++n) {
                    const int slot = n % STAGES;
                    i4::copy_wait<CODE_DEPTH - 2>();
                    ok = __all_sync(0xFFFFFFFFu, wait(&sm.done[slot], ((n / STAGES) & 1u) ^ 1u));
                    if (!ok) break;
                    tc::tc_fence_after();
                    __syncwarp();                // the other lanes' copies (zero points)
                    copy_next();
#pragma unroll
                    for (int tile = 0; tile < STAGE_TILES; ++tile) {
                        uint32_t r[16], v[4];
                        if (2 * st + tile < c.kt) {
                            const uint4 code = sm.codes[w][at][tile][lane];
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const uint32_t z = c.z ? sm.zeros[w][at][tile * 2 + half][g] : I4_ZERO;
                                i4::widen(half ? code.y : code.x, __byte_perm(z, 0, 0x1010), v);
                                r[8 * half] = v[0], r[8 * half + 1] = v[1], r[8 * half + 4] = v[2], r[8 * half + 5] = v[3];
                                i4::widen(half ? code.w : code.z, __byte_perm(z, 0, 0x3232), v);
                                r[8 * half + 2] = v[0], r[8 * half + 3] = v[1], r[8 * half + 6] = v[2], r[8 * half + 7] = v[3];
                            }
                        } else {                 // channels past the image
#pragma unroll
                            for (int i = 0; i < 16; ++i) r[i] = 0u;
                        }
                        tmem_st_16x32(to + slot * A_COLS + tile * (A_COLS / STAGE_TILES), r);
                    }
                    at = at + 1 == CODE_DEPTH ? 0 : at + 1;
                    tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.full[slot]);
                }
            }
            i4::copy_wait<0>();
        } else if (warp < DRAIN_WARPS + WIDEN_WARPS + LOAD_WARPS) {
            // ------------------------------------------------------------ rows of x into shared memory
            const int tid = threadIdx.x - (DRAIN_WARPS + WIDEN_WARPS) * 32, lw = tid >> 5;
            constexpr int STEP = LOAD_WARPS * 4;             // rows that the threads cover at once, 8 chunks each
            constexpr int PER = (S::BN + STEP - 1) / STEP;
            const int chunk = tid & 7, r0 = tid >> 3;
            uint32_t n = 0, arrived = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const i4::Unit un = unit_at(u);
                int src[PER];
                if (c.x_grid == 16) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int r = r0 + i * STEP;
                        src[i] = r < un.count ? i4::source_row(c, un.row0 + r) : -1;
                    }
                }
                for (int st = 0; st < stages; ++st, ++n) {
                    const int slot = n % STAGES;
                    ok = __all_sync(0xFFFFFFFFu, wait(&sm.done[slot], ((n / STAGES) & 1u) ^ 1u));
                    if (!ok) break;
                    if (c.x_grid == 16) {
                        const int k = st * STAGE_K + chunk * 8;
                        const uint32_t base = smem_addr(sm.x[slot][0]) + ((chunk ^ (r0 & 7)) << 4) + r0 * 128;
                        const int have0 = min(max(c.K - k, 0), 8) * 2, have1 = min(max(c.K - k - I4_K, 0), 8) * 2;
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            if (r0 + i * STEP >= un.count) break;
                            // the swizzle of rows r0 + 12 i: 12 i changes r & 7 by 4 for odd i
                            const uint32_t to = (base + i * STEP * 128) ^ ((i & 1) << 6);
                            const uint16_t* from = c.x + (src[i] < 0 ? 0 : src[i]) * c.ldx + k;
                            const int b0 = src[i] < 0 ? 0 : have0, b1 = src[i] < 0 ? 0 : have1;
                            i4::copy16(to, b0 ? from : c.x, b0);
                            i4::copy16(to + S::BN * 128, b1 ? from + I4_K : c.x, b1);
                        }
                    } else {
                        // rows off the 16-byte grid: a warp takes a row, two channels a lane, eight rows at a time
                        constexpr int BATCH = 8;
#pragma unroll 1
                        for (int rb = lw; rb < un.count; rb += LOAD_WARPS * BATCH) {
#pragma unroll 1
                            for (int tile = 0; tile < STAGE_TILES; ++tile) {
                                const int k = (st * STAGE_TILES + tile) * I4_K + lane * 2;
                                uint32_t v[BATCH];
#pragma unroll
                                for (int i = 0; i < BATCH; ++i) {
                                    const int r = rb + i * LOAD_WARPS;
                                    const int from = r < un.count ? i4::source_row(c, un.row0 + r) : -1;
                                    const uint16_t* p = c.x + (from < 0 ? 0 : from) * c.ldx + k;
                                    const uint32_t lo = from >= 0 && k < c.K ? p[0] : 0u, hi = from >= 0 && k + 1 < c.K ? p[1] : 0u;
                                    v[i] = lo | hi << 16;
                                }
#pragma unroll
                                for (int i = 0; i < BATCH; ++i) {
                                    const int r = rb + i * LOAD_WARPS;
                                    if (r < un.count)
                                        *reinterpret_cast<uint32_t*>(sm.x[slot][tile] + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4) = v[i];
                                }
                            }
                        }
                    }
                    i4::copy_commit();
                    if (n >= LOAD_LAG) {
                        i4::copy_wait<LOAD_LAG>();
                        fence_async_proxy();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.full[arrived % STAGES]);
                        ++arrived;
                    }
                }
            }
            i4::copy_wait<0>();
            fence_async_proxy();
            __syncwarp();
            for (; arrived < n; ++arrived)
                if (lane == 0) mbar_arrive(&sm.full[arrived % STAGES]);
        } else if (lane == 0) {
            // ------------------------------------------------------------ MMA issuer
            uint32_t n = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const i4::Unit un = unit_at(u);
                const uint32_t idesc = idesc_for((un.count + 15) / 16 * 16);
                for (int st = 0; st < stages; ++st, ++n) {
                    const int slot = n % STAGES;
                    ok = wait(&sm.drained[n & 1], ((n >> 1) & 1u) ^ 1u) && wait(&sm.full[slot], (n / STAGES) & 1u);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint32_t a = tmem + A_BASE + slot * A_COLS;
#pragma unroll
                    for (int k = 0; k < STAGE_K / 16; ++k) {
                        const uint32_t d = tmem + (n & 1) * COLS + k / (8 / CHUNKS) * S::BN;
                        const uint64_t b = tc::sw128_desc(smem_addr(sm.x[slot][k / 4])) + 2 * (k % 4);
                        mma_ts(d, a + k * 8, b, idesc, k % (8 / CHUNKS) != 0);
                    }
                    tc::mma_commit(&sm.done[slot]);
                }
            }
            // every issued MMA must complete before the tensor memory is released
            if (n) {
                tc::mma_commit(&sm.last);
                mbar_wait_bounded(&sm.last, 0u, LANDING_LIMIT, c.status, nullptr);
            }
        }
    } else {
        // ---------------------------------------------------------------- drain, scale, add up
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(DRAIN_REGS));
        constexpr int PIECES = S::BN / 32;                   // 16-column pieces per thread: every second one
        const int quarter = warp & 3, side = warp >> 2;
        const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + side * 16;
        const int row = quarter * 32 + lane, block = row >> 4, g = row & 7, upper = (row >> 3) & 1;
        int p_unit = blockIdx.x, p_stage = 0, p_slot = 0;
        size_t p_rec = 0;
        bool p_have = false;
        auto enter = [&](int u) {
            const i4::Unit un = unit_at(u);
            const int b = un.tile * BM_BLOCKS + block;
            p_have = b < c.blocks;
            p_rec = ((size_t)un.expert * c.blocks + b) * c.groups * 8 + g;
        };
        auto copy_next = [&]() {
            if (p_unit < units) {
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) {
                    const int step = p_stage * 4 + j * (4 / CHUNKS);
                    if (p_have && step < 2 * c.kt) {
                        const size_t rec = p_rec + (size_t)i4::group_of(c, step) * 8;
                        i4::copy_small<4>(smem_addr(&sm.scales[p_slot][j][threadIdx.x]),
                                          c.s_f32 ? c.s + rec * 8 + upper * 4 : c.s + rec * 4);
                    }
                }
                if (++p_stage == stages) {
                    p_stage = 0;
                    p_unit += gridDim.x;
                    if (p_unit < units) enter(p_unit);
                }
            }
            p_slot = (p_slot + 1) % SCALE_DEPTH;
            i4::copy_commit();
        };
        if (p_unit < units) enter(p_unit);
#pragma unroll 1
        for (int i = 0; i < SCALE_DEPTH - 1; ++i) copy_next();
        uint32_t n = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const i4::Unit un = unit_at(u);
            float acc[PIECES][16];
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[p][i] = 0.f;
            for (int st = 0; st < stages; ++st, ++n) {
                const int slot = n % STAGES;
                i4::copy_wait<SCALE_DEPTH - 2>();
                copy_next();
                float sc[CHUNKS];
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) {
                    const uint32_t v = sm.scales[n % SCALE_DEPTH][j][threadIdx.x];
                    sc[j] = __uint_as_float(c.s_f32 ? v : upper ? v & 0xFFFF0000u : v << 16);
                    // the last stage's second tile may lie past the matrix
                    if (st * 4 + j * (4 / CHUNKS) >= 2 * c.kt) sc[j] = 0.f;
                }
                ok = __all_sync(0xFFFFFFFFu, wait(&sm.done[slot], (n / STAGES) & 1u));   // tcgen05.ld below is warp-collective
                if (!ok) break;
                tc::tc_fence_after();
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
                    for (int p = 0; p < PIECES; ++p)
                        if (p * 32 + side * 16 < un.count) {
                            uint32_t part[16];
                            tc::tmem_ld16u(from + (n & 1) * COLS + j * S::BN + p * 32, part);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; i += 2) tc::fma2(acc[p][i], acc[p][i + 1], part[i], part[i + 1], sc[j]);
                        }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.drained[n & 1]);
            }
            if (!ok) break;
            const int n0 = c.gated ? (un.tile * BM_BLOCKS + block) * 8 + g : un.tile * 128 + row;
            const bool mine = n0 < c.N && !(c.gated && upper);
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int m = p * 32 + side * 16 + i;
                    float v = acc[p][i];
                    if (c.gated) {
                        const float up = __shfl_xor_sync(0xFFFFFFFFu, v, 8);
                        v = i4::gate(v, up);
                    }
                    if (mine && m < un.count) i4::store_y(c, un.row0 + m, n0, v);
                }
        }
        i4::copy_wait<0>();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

template <int CHUNKS>
cudaError_t launch(const moe_int4* L, const Int4Call& c, cudaStream_t s) {
    constexpr int fixed = sizeof(Smem<CHUNKS>) + 1024;
    constexpr int most = fixed + 2 * (MOE_DISPATCH_MAX_EXPERTS + 1) * (int)sizeof(int);
    static_assert(most <= 227 * 1024 - 1024, "shared memory");
    cudaError_t e = ensure_smem_limit<int4_many_kernel<CHUNKS>>(most);
    if (e != cudaSuccess) return e;
    const int bn = Smem<CHUNKS>::BN;
    const int64_t tiles = (c.blocks + BM_BLOCKS - 1) / BM_BLOCKS;
    const int64_t row_tiles = c.offsets ? std::min<int64_t>(c.rows, c.rows / bn + c.E) : (c.rows + bn - 1) / bn;
    const int64_t grid = std::min<int64_t>(tiles * row_tiles, L->num_sms);
    return launch_pdl(int4_many_kernel<CHUNKS>, dim3((unsigned)grid), dim3(NTHREADS), fixed + 2 * (c.E + 1) * (int)sizeof(int), s, c, bn);
}

}  // namespace

bool int4_takes_many(const Int4Call& c) { return (c.offsets ? c.rows / c.E : c.rows) > 32; }

cudaError_t launch_int4_many(const moe_int4* L, const Int4Call& c, cudaStream_t s) {
    const int group = L->d.group;
    if (group % 128 == 0 || L->groups == 1) return launch<1>(L, c, s);
    return group % 64 == 0 ? launch<2>(L, c, s) : launch<4>(L, c, s);
}

}  // namespace moe
