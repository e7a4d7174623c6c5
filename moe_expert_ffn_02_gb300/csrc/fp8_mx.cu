// FP8 projections of many tokens with e8m0 scales, plain and gated: the tensor
// core applies the scales itself (tcgen05.mma kind::mxf8f6f4, block_scale), so
// a whole K range accumulates in tensor memory and is drained once.
//
// Bound by the SM: a K block's 48 KB are written to shared memory and read by the MMAs in about 680 cycles,
// 512 of them MMA work (0.355 us a block with 19 CTAs as with 152).  The fp32-scale form has to drain and scale 128 x 256
// partial sums for every 512 cycles of MMA work (about 780 in all); here a tile
// costs its MMAs plus one drain: 4096 x 7168 x 7168 131 us (3.2 PFLOP/s, 0.85 of twice the bf16 rate),
// gated 8192 x 7168 x 2048 144 us (0.89); the tensor pipe is busy 70 and 73 % of the time.  The hardware takes one power-of-two factor per
// row and 32 channels: the four K32 steps of a 128-channel block use the same
// byte, and the four bytes of a 32-bit word hold four consecutive K blocks (a
// quad), selected by the instruction's scale-factor id.
//
// The accumulator is fp32 and truncates: each MMA loses up to one unit in the
// last place of the running sum at that point, always towards zero, so a chain is
// limited to MAX_KT blocks: 256 MMAs lose below 256 x 2^-23 of the largest partial
// sum, which sums that cancel later may leave far behind (in terms of the result
// there is no bound), and operands of one sign lose all in the same direction
// (2100 x 8192 x 2100, chains of 64 blocks: 5e-6 of the sum; fp32 scales 6e-7).
// Longer ones take the form that adds blocks in registers, each sum rounded.
//
// Scale factors reach tensor memory through shared memory (tcgen05.cp
// 32x128b.warpx4): 128 rows x 4 K blocks in 512 bytes, row r at (r mod 32) * 16 +
// (r / 32) * 4.  The weights' are laid out so once; the tokens' come as four rows
// of bytes, which warp 2 transposes.
//
// Warps as in the fp32-scale form.  BN = 256: one accumulator of 256 columns, read
// into registers (128 a thread) and handed back before the epilogue's arithmetic
// and stores, which the next tile's MMAs cover; BN = 128: two accumulators.
#include "fp8_gemm.cuh"

namespace moe {
namespace mx {

using namespace dg;

constexpr int MAX_KT = 64;
constexpr int SF_SLOTS = 3;
constexpr int RAW_BYTES = 4 * BM;                        // tokens' bytes of a quad, [4 K blocks][128 rows]
constexpr int SF_BYTES = 512;                            // packed: 128 rows x 4 K blocks

template <int BN>
constexpr int slot_bytes() { return RAW_BYTES + SF_BYTES + BN / QB * SF_BYTES; }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

template <int BN, bool GATED>
__global__ void __launch_bounds__(NTHREADS, 1) mx_kernel(const __grid_constant__ Maps maps, const uint8_t* __restrict__ wsf, int nrb,
                                                        Args a) {
    constexpr int HALF = BN / 2, NBUF = BUF_COLS / BN;
    constexpr int SF_COL = BUF_COLS;                     // scale factors lie behind the accumulators: 2 slots of 16 columns
    constexpr int SLOT = slot_bytes<BN>();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int w_bytes = BN * 128;
    const int a_bytes = a.a_rows * 128, stage_bytes = w_bytes + a_bytes;
    uint8_t* tail = ring + a.stages * stage_bytes;
    float* amax_cta = reinterpret_cast<float*>(tail);
    uint8_t* sf = tail + (GATED ? TAIL_GATED : TAIL_PLAIN);                     // [SF_SLOTS][raw | tokens | weights]
    __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[NBUF], tempty[NBUF], xbar[2];
    __shared__ uint64_t sfull[SF_SLOTS], sready[SF_SLOTS], sempty[SF_SLOTS], mma_done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a cluster shares a unit's K (S > 1), or the 128 features of a gated unit
    constexpr bool CAN_SPLIT = !GATED || BN == 256;
    const bool shared_k = CAN_SPLIT && a.S > 1;
    const uint32_t crank = cluster_rank(), cctas = cluster_size();
    const uint32_t rank = shared_k ? 0u : crank, csize = shared_k ? 1u : cctas;
    const int first = blockIdx.x / cctas, step = gridDim.x / cctas;
    // this CTA's K blocks [kb0, kb0 + kt): whole quads
    const int quads = (a.kt + 3) / 4, split = shared_k ? (int)crank : 0;
    const int kb0 = quads * split / a.S * 4, kt = min(a.kt, quads * (split + 1) / a.S * 4) - kb0;

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        for (int b = 0; b < NBUF; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], EPI_WARPS); }
        for (int b = 0; b < SF_SLOTS; ++b) { mbar_init(&sfull[b], 1); mbar_init(&sready[b], 1); mbar_init(&sempty[b], 1); }
        for (int b = 0; b < 2; ++b) mbar_init(&xbar[b], 1);
        mbar_init(&mma_done, 1);
        fence_mbar_init();
        abort_flag = 0;
    }
    __syncthreads();
    if (GATED && csize > 1) cluster_arrive();
    volatile int* abort = &abort_flag;

    auto unit_rows = [&](int u, int& m0, int& n0) {
        const int mt = u / a.n_nt;
        m0 = mt * BM;
        n0 = ((u - mt * a.n_nt) * (int)csize + (int)rank) * BN;
    };

    if (warp < CTRL_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTRL_REGS));
        if (warp == 0) {
            // ------------------------------------------------ producer
            const uint32_t el = elect_one();
            const uint32_t ring0 = smem_addr(ring), full0 = smem_addr(full), sf0 = smem_addr(sf), sfull0 = smem_addr(sfull);
            if (el) {
                prefetch_map(&maps.w);
                prefetch_map(&maps.a);
                prefetch_map(&maps.s);
            }
            int stage = 0, slot = 0;
            uint32_t phase = 0, sphase = 0;
            int issued = 0, sissued = 0;
            bool ok = true;
            pdl_wait();
            for (int u = first; u < a.n_units && ok; u += step) {
                int m0, n0;
                unit_rows(u, m0, n0);
                // 128-row scale blocks of the tile that exist (a cluster's last tiles may lie past the image)
                const int blocks = max(0, min(BN / QB, nrb - n0 / QB));
                for (int kb = 0; kb < kt; ++kb) {
                    if ((kb & 3) == 0) {
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&sempty[slot], sphase ^ 1u, a.wait_limit, a.status, abort));
                        if (!ok) break;
                        if (el) {
                            expect_tx(sfull0 + 8 * slot, (uint32_t)(RAW_BYTES + blocks * SF_BYTES));
                            tma_load_2d(sf0 + slot * SLOT, &maps.s, m0, kb0 + kb, sfull0 + 8 * slot);
                            if (blocks > 0)
                                bulk_g2s(sf + slot * SLOT + RAW_BYTES + SF_BYTES,
                                         wsf + ((size_t)((kb0 + kb) >> 2) * nrb + n0 / QB) * SF_BYTES, (uint32_t)(blocks * SF_BYTES),
                                         &sfull[slot]);
                        }
                        sissued = min(sissued + 1, SF_SLOTS);
                        if (++slot == SF_SLOTS) { slot = 0; sphase ^= 1u; }
                    }
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[stage], phase ^ 1u, a.wait_limit, a.status, abort));
                    if (!ok) break;
                    if (el) {
                        const uint32_t dst = ring0 + stage * stage_bytes, bar = full0 + 8 * stage;
                        expect_tx(bar, (uint32_t)stage_bytes);
                        tma_load_3d(dst, &maps.w, 0, n0, kb0 + kb, bar);
                        copy_tokens(maps, a.k_full, a.kt, dst + w_bytes, kb0 + kb, 1, m0, a_bytes, bar);
                    }
                    issued = min(issued + 1, a.stages);
                    if (++stage == a.stages) { stage = 0; phase ^= 1u; }
                }
            }
            for (; issued > 0; --issued) {                 // every issued copy lands before the CTA exits
                if (--stage < 0) { stage = a.stages - 1; phase ^= 1u; }
                mbar_wait_bounded(&full[stage], phase, LANDING_LIMIT_US, a.status, nullptr);
            }
            for (; sissued > 0; --sissued) {
                if (--slot < 0) { slot = SF_SLOTS - 1; sphase ^= 1u; }
                mbar_wait_bounded(&sfull[slot], sphase, LANDING_LIMIT_US, a.status, nullptr);
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issuer
            tc::tmem_alloc(&tmem_slot, 512);
            tc::tc_fence_before();
            named_bar_sync(2, (1 + EPI_WARPS) * 32);
            tc::tc_fence_after();
            pdl_wait();                                    // no bounded wait before it
            const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_slot, 0);
            const uint32_t el = elect_one();
            const uint32_t d0 = (uint32_t)tc::sw128_desc(smem_addr(ring)), sf0 = smem_addr(sf);
            int stage = 0, slot = 0, tslot = 0, buf = 0;
            uint32_t phase = 0, sphase = 0, tphase = 0;
            bool ok = true, issued = false;
            const int stop = a.plant && blockIdx.x == 0 ? kt - 1 : -1;
            for (int u = first; u < a.n_units && ok; u += step) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&tempty[buf], tphase ^ 1u, a.wait_limit, a.status, abort));
                const uint32_t dt = tmem + (uint32_t)(buf * BN);
                for (int kb = 0; kb < kt && ok; ++kb) {
                    const uint32_t sft = tmem + SF_COL + (uint32_t)(tslot * 16);
                    if ((kb & 3) == 0) {
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&sready[slot], sphase, a.wait_limit, a.status, abort) &&
                                                         mbar_wait_bounded(&sfull[slot], sphase, a.wait_limit, a.status, abort));
                        if (!ok) break;
                        issued = true;
                        const uint32_t at = sf0 + slot * SLOT + RAW_BYTES;
                        sf_copy(sft, sf_desc(at), el);
#pragma unroll
                        for (int b = 0; b < BN / QB; ++b) sf_copy(sft + 4 + 4 * b, sf_desc(at + SF_BYTES * (1 + b)), el);
                    }
                    ok = kb != stop && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[stage], phase, a.wait_limit, a.status, abort));
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint32_t wd = d0 + (uint32_t)((stage * stage_bytes) >> 4), ad = wd + (uint32_t)(w_bytes >> 4);
                    const uint32_t idesc = idesc_mx(BN, kb & 3);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_mx(dt, ad + 2 * k, wd + 2 * k, idesc, sft, sft + 4, (kb | k) != 0, el);
                    const bool quad_end = (kb & 3) == 3 || kb == kt - 1;
                    if (el) {
                        tc::mma_commit(&empty[stage]);
                        if (quad_end) tc::mma_commit(&sempty[slot]);
                        if (kb == kt - 1) tc::mma_commit(&tfull[buf]);
                    }
                    __syncwarp();
                    if (quad_end) {
                        if (++slot == SF_SLOTS) { slot = 0; sphase ^= 1u; }
                        tslot ^= 1;
                    }
                    if (++stage == a.stages) { stage = 0; phase ^= 1u; }
                }
                if (++buf == NBUF) { buf = 0; tphase ^= 1u; }
            }
            if (!ok && issued) finish_mmas(&mma_done, el, a.status);
        } else if (warp == 2) {
            // ------------------------------------------------ tokens' scale factors: [4 K blocks][row] -> [row][4 K blocks]
            int slot = 0;
            uint32_t sphase = 0;
            bool ok = true;
            pdl_wait();
            for (int u = first; u < a.n_units && ok; u += step) {
                for (int q = 0; q < (kt + 3) / 4; ++q) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&sfull[slot], sphase, a.wait_limit, a.status, abort));
                    if (!ok) break;
                    const uint32_t* raw = reinterpret_cast<const uint32_t*>(sf + slot * SLOT);
                    uint32_t* dst = reinterpret_cast<uint32_t*>(sf + slot * SLOT + RAW_BYTES);
                    const uint32_t w0 = raw[lane], w1 = raw[32 + lane], w2 = raw[64 + lane], w3 = raw[96 + lane];
                    const uint32_t lo01 = prmt(w0, w1, 0x5140), lo23 = prmt(w2, w3, 0x5140);      // rows 4 lane, + 1
                    const uint32_t hi01 = prmt(w0, w1, 0x7362), hi23 = prmt(w2, w3, 0x7362);      // rows + 2, + 3
                    const int r = 4 * lane, at = (r & 31) * 4 + (r >> 5);                         // in words; next row 4 further
                    dst[at] = prmt(lo01, lo23, 0x5410);
                    dst[at + 4] = prmt(lo01, lo23, 0x7632);
                    dst[at + 8] = prmt(hi01, hi23, 0x5410);
                    dst[at + 12] = prmt(hi01, hi23, 0x7632);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sready[slot]);
                    if (++slot == SF_SLOTS) { slot = 0; sphase ^= 1u; }
                }
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        // ---------------------------------------------------- drain warps
        const int ew = warp - CTRL_WARPS, quarter = warp & 3, half = ew >> 2;
        named_bar_sync(2, (1 + EPI_WARPS) * 32);
        tc::tc_fence_after();
        const uint32_t tmem = tmem_slot + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * HALF);
        pdl_wait();
        if (GATED && csize > 1) cluster_wait();
        EpiCtx ctx = {ew, quarter, half, lane, rank, csize, staging<false>(tail, GATED, ew), amax_cta,
                      amax_cta + 2 * BM, xbar, 0, 0u, abort};
        int buf = 0;
        uint32_t tphase = 0;
        bool dead = false;
        for (int u = first; u < a.n_units; u += step) {
            int m0, n0;
            unit_rows(u, m0, n0);
            const int valid = min(BM, a.M - m0);
            const bool live = quarter * 32 < valid;
            float acc[HALF];
            if (!dead && !mbar_wait_bounded(&tfull[buf], tphase, a.wait_limit, a.status, abort)) dead = true;
            dead = __any_sync(0xFFFFFFFFu, dead);
            if (live && !dead) {
                tc::tc_fence_after();
#pragma unroll
                for (int c = 0; c < HALF; c += 32)
                    tc::tmem_ld32u(tmem + (uint32_t)(buf * BN + c), reinterpret_cast<uint32_t(&)[32]>(acc[c]));
                tc::tmem_wait_ld();
                tc::tc_fence_before();
            } else {
#pragma unroll
                for (int c = 0; c < HALF; ++c) acc[c] = 0.f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
            if (++buf == NBUF) { buf = 0; tphase ^= 1u; }
            if constexpr (CAN_SPLIT) {
                if (shared_k) {
                    if (live) leave_partial<HALF>(reinterpret_cast<float*>(ring), half, quarter * 32 + lane, acc);
                    tell_peers(dead, abort, a.S, lane);
                    cluster_arrive_release();
                    cluster_wait();
                    if (!*abort) join_partials<BN, GATED>(a, smem_addr(ring), split, ew, lane, m0, n0, valid);
                    continue;
                }
            }
            if constexpr (GATED) epi_gated<HALF>(a, ctx, acc, m0, n0, valid, dead);
            else if (live && !dead) epi_plain<HALF, false>(maps.y, a, ctx, acc, m0, n0, valid);
        }
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

template <int BN, bool GATED>
cudaError_t launch_mx(const GemmCall& c, Args& a, int S, cudaStream_t s) {
    const moe_linear* L = c.lin;
    const int cluster = S > 1 ? S : GATED ? BUF_COLS / BN : 1;
    a.S = S;
    const int mt = (c.M + BM - 1) / BM;
    a.bn = BN;
    a.n_nt = GATED ? (L->d.out_features + QB - 1) / QB : (L->rows + BN - 1) / BN;
    const long long units = (long long)mt * a.n_nt;
    if (units > 0x3FFFFFFF) return cudaErrorInvalidValue;
    a.n_units = (int)units;
    Maps maps;
    if (!encode_maps(c, a, 1, BM, 4, &maps)) return cudaErrorInvalidValue;       // scales: a quad of 128 rows
    const int stage = (BN + a.a_rows) * 128, fixed = 1024 + (GATED ? TAIL_GATED : TAIL_PLAIN) + SF_SLOTS * slot_bytes<BN>();
    a.stages = std::min(MAX_STAGES, (SMEM_MAX - fixed) / stage);
    if (S > 1 && a.stages * stage < BM * part_pitch(BN) * 4) return cudaErrorInvalidValue;
    cudaError_t e = ensure_smem_limit<mx_kernel<BN, GATED>>(SMEM_MAX);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = fixed + a.stages * stage;
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
    cfg.gridDim = dim3((unsigned)((S > 1 ? units : std::min<long long>(units, L->num_sms / cluster)) * cluster));
    return cudaLaunchKernelEx(&cfg, mx_kernel<BN, GATED>, maps, (const uint8_t*)L->wsf, (L->rows_pad + QB - 1) / QB, a);
}

}  // namespace mx

MxPlan plan_fp8_mx(const GemmCall& c, bool gated) {
    using namespace dg;
    MxPlan best = {};
    const Args a = base_args(c);
    if (!c.lin->wsf || a.kt > mx::MAX_KT) return best;
    // A tile's K block takes its MMAs (512 cycles for 256 rows, half for 128) or its copies.  256 rows
    // reuse the tokens best; 128 rows, or K split over S CTAs, use SMs that tiles alone leave idle.
    const int sms = c.lin->num_sms, quads = (a.kt + 3) / 4;
    const double mt = (c.M + BM - 1) / BM;
    const double rows = gated ? 2.0 * ((c.lin->d.out_features + QB - 1) / QB * QB) : (double)c.lin->rows;
    for (int b = 128; b <= 256; b += 128) {
        const double units = mt * std::ceil(rows / b), kb = std::max(b / 256.0 * 0.257, copy_us(b, a.a_rows));
        for (int k = 1; k <= 8 && k <= quads; k *= 2) {
            if (k > 1 && (units > cluster_slots(sms, k) || (gated && b == 128))) break;
            const double kr = std::min<double>(a.kt, 4.0 * ((quads + k - 1) / k));
            const double us = plan_us(k > 1 ? 1.0 : std::ceil(units / sms), kr, kb, 0.734 + 0.19 * b / 256 + (gated ? 0.69 : 0.0), memory_bytes(c, gated)) +
                              join_us(gated, b, k, c.M, units * k) + (gated && b == 128 ? 0.126 : 0.0);
            if (best.bn == 0 || us < best.us) best = MxPlan{b, k, us};
        }
    }
    return best;
}

cudaError_t launch_fp8_mx(const GemmCall& c, bool gated, const MxPlan& p, cudaStream_t s) {
    using namespace dg;
    Args a = base_args(c);
    if (p.bn == 128) return gated ? mx::launch_mx<128, true>(c, a, p.S, s) : mx::launch_mx<128, false>(c, a, p.S, s);
    return gated ? mx::launch_mx<256, true>(c, a, p.S, s) : mx::launch_mx<256, false>(c, a, p.S, s);
}

}  // namespace moe
