// The mx (ue8m0 scales per 32 k) instances of the 4-bit floating-point GEMM, and
// the plan that both formats share.
#include "gemm_fp4.cuh"

namespace igemm {

int fp4_plan(const Fp4Call &c, int (*max_clusters)(int, bool, int), Fp4Plan *plan)
{
    const int blocks = (c.K + 511) / 512;
    // activation rows of a typical group, and the groups that have any
    double groups = 1.0;
    if (c.offsets) groups = c.experts * (1.0 - std::pow(1.0 - 1.0 / c.experts, double(c.rows)));
    const double typical = c.rows / groups;
    plan->cs = 1;
    plan->pair = false;
    plan->bn = typical <= 16 ? 16 : typical <= 32 ? 32 : typical <= 64 ? 64 : 128;
    if (typical > 128) {
        const double slots = double((c.N + 255) / 256) * std::ceil(typical / 256) * groups;
        if (slots * 2 >= sm_count() / 2) {
            plan->pair = true;
            plan->bn = 256;
        }
    }
    plan->qt = plan->bn;
    const int64_t p_tiles = (c.N + (plan->pair ? 255 : 127)) / (plan->pair ? 256 : 128);
    // a group's weights (32 MB of codes) stay in L2 while it runs
    const int64_t slot_bytes = int64_t(plan->pair ? 256 : 128) * fp4_code_bytes(c.K);
    plan->group_p = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(p_tiles, (int64_t(32) << 20) / slot_bytes)));
    if (plan->pair) return kOk;
    const double tiles = double(p_tiles) * std::ceil(typical / plan->bn) * groups;
    double best = -1;
    for (int cs = 1; cs <= (plan->bn == 128 ? 2 : plan->bn == 16 ? 4 : 8); cs *= 2) {
        const int per = (blocks + cs - 1) / cs;
        if (cs > 1 && per * (cs - 1) >= blocks) break;
        const int clusters = max_clusters(plan->bn, false, cs);
        if (clusters < 1) return kCudaError;
        // the busiest cluster's stages, plus a tile's fill and epilogue
        const double cost = std::ceil(tiles / clusters) * (per + (cs > 1 ? 1.5 : 1.0));
        if (best < 0 || cost < best) {
            best = cost;
            plan->cs = cs;
        }
    }
    return kOk;
}

int launch_fp4_mx(const Fp4Call &c, cudaStream_t stream) { return launch_fp4_format<false>(c, stream); }

}  // namespace igemm
