// Gated FP8 projection h = SiLU(A Wg^T) * (A Wu^T), quantised to 1x128 E4M3
// in the GEMM's epilogue, so the two fp32 products never leave the SM.
//
// A unit is 128 tokens x 128 features: 256 interleaved gate/up rows, in one
// CTA or split over a cluster of 2 or 4 CTAs, or its K over 2, 4 or 8.  The CTAs of a cluster exchange
// their rows' amax through distributed shared memory before they quantise.
// Bound like the plain one; the epilogue of a unit (SiLU's exponential and quotient,
// two special-function operations a feature: 2000 cycles) is not covered by the next
// unit's MMAs beyond two K blocks: 7 x 4300 cycles of 196 us at 8192 x 7168 x 2048.
#include "fp8_gemm.cuh"

namespace moe {
namespace dg {

// CTAs per unit of 128 features: a cluster that shares its rows, or its K.
static Plan plan_gated(const GemmCall& c, const Args& a) {
    const int sms = c.lin->num_sms;
    const int mt = (c.M + BM - 1) / BM, nt = (c.lin->d.out_features + QB - 1) / QB;
    const long long units = (long long)mt * nt;
    Plan best = {};
    double best_us = 0;
    if (units > 0x3FFFFFFF) return best;
    // a unit's K block takes the draining of its columns, or its copies
    auto block_us = [&](int grp, int bn) {
        return std::max(grp == 1 ? 0.46 : grp == 2 ? 0.305 : 0.098, copy_us(bn, a.a_rows));
    };
    auto fixed_us = [](int bn) { return 1.635 + 0.447 * bn / 256; };
    const double bytes = memory_bytes(c, true);
    for (int cl = 1; cl <= MAX_CLUSTER; cl *= 2) {
        const int grp = cl, bn = BUF_COLS / cl, slots = cluster_slots(sms, cl);
        // rows over eight CTAs: two stages of eight K blocks do not fit beside 72 token rows and more
        if (cl <= 4) {
            const double us = plan_us((double)((units + slots - 1) / slots), a.kt, block_us(grp, bn), fixed_us(bn), bytes) +
                              (cl > 1 ? 0.126 : 0.0);
            if (best.bn == 0 || us < best_us) {
                best_us = us;
                best = Plan{grp, bn, cl, (int)units, nt, 1, us};
            }
        }
        if (cl > 1 && cl <= a.kt && units <= slots) {
            const double us = plan_us(1.0, (a.kt + cl - 1) / cl, block_us(1, BUF_COLS), fixed_us(BUF_COLS), bytes) +
                              join_us(true, BUF_COLS, cl, c.M, (double)units * cl);
            if (best.bn == 0 || us < best_us) {
                best_us = us;
                best = Plan{1, BUF_COLS, cl, (int)units, nt, cl, us};
            }
        }
    }
    return best;
}

}  // namespace dg

cudaError_t launch_fp8_gated(const GemmCall& c, cudaStream_t s) {
    using namespace dg;
    if (few_tokens(c)) return launch_fp8_few(c, true, s);
    Args a = base_args(c);
    const Plan p = plan_gated(c, a);
    if (!p.bn) return cudaErrorInvalidValue;
    const MxPlan mx = plan_fp8_mx(c, true);
    if (mx.bn && mx.us <= p.us) return launch_fp8_mx(c, true, mx, s);
    switch (p.grp) {
        case 1: return launch<1, true>(c, p, a, s);
        case 2: return launch<2, true>(c, p, a, s);
        default: return launch<4, true>(c, p, a, s);
    }
}

}  // namespace moe
