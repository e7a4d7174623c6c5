// Gated FP8 projection h = SiLU(A Wg^T) * (A Wu^T), quantised to 1x128 E4M3
// in the GEMM's epilogue, so the two fp32 products never leave the SM.
//
// A unit is 128 tokens x 128 features: 256 interleaved gate/up rows, in one
// CTA or split over a cluster of 2, 4 or 8 CTAs.  The CTAs of a cluster exchange
// their rows' amax through distributed shared memory before they quantise.
#include "fp8_gemm.cuh"

namespace moe {
namespace dg {

static Plan plan_gated(const GemmCall& c, const Args& a) {
    const int sms = c.lin->num_sms;
    const int mt = (c.M + BM - 1) / BM, nt = (c.lin->d.out_features + QB - 1) / QB;
    Plan best = {};
    double best_cost = 0;
    for (int cl = 1; cl <= MAX_CLUSTER; cl *= 2) {
        const int grp = cl, bn = BUF_COLS / cl;
        if (2 * stage_cost(grp, bn, a.a_rows, a.e8m0) > ring_max(true)) continue;
        const long long units = (long long)mt * nt;
        if (units > 0x3FFFFFFF) continue;
        const int slots = sms / cl;
        const double waves = (double)((units + slots - 1) / slots);
        const double drain = grp == 1 ? 1000 : grp == 2 ? 560 : grp == 4 ? 300 : 180;
        const double share = (double)(units < slots ? units : slots) * cl;
        const double hbm = mt == 1 ? bn * 128.0 * share / 3600.0 : 0.0;
        const double l2 = (bn + a.a_rows) * 128.0 / 60.0;
        const double per = std::max(drain, std::max(hbm, l2));
        const double cost = waves * (a.kt * per + 3000.0 + (cl > 1 ? 1500.0 : 0.0));
        if (best.bn == 0 || cost < best_cost) {
            best_cost = cost;
            best = Plan{grp, bn, cl, (int)units, nt};
        }
    }
    return best;
}

}  // namespace dg

cudaError_t launch_fp8_gated(const GemmCall& c, cudaStream_t s) {
    using namespace dg;
    if (few_tokens(c, true)) return launch_fp8_few(c, true, s);
    if (mx_fits(c.lin)) return launch_fp8_mx(c, true, s);
    Args a = base_args(c);
    a.hq = c.hq;
    a.ld_hq = c.ld_hq;
    a.hs = c.hs;
    a.ld_hs = c.ld_hs;
    const Plan p = plan_gated(c, a);
    if (!p.bn) return cudaErrorInvalidValue;
    switch (p.grp) {
        case 1: return launch<1, true>(c, p, a, s);
        case 2: return launch<2, true>(c, p, a, s);
        case 4: return launch<4, true>(c, p, a, s);
        default: return launch<8, true>(c, p, a, s);
    }
}

}  // namespace moe
