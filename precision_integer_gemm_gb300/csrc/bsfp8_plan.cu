// Host only: the kernel, tile and split of a block-scaled fp8 product.
#include <algorithm>
#include <cmath>
#include "bsfp8.cuh"

namespace igemm {

// Kernel, tile and split by estimated time in microseconds.  A wave of tiles takes
// groups of 512 k times the time of a group on an SM: what its bytes take from L2 (100
// KB a microsecond) or from HBM (6.3 MB a microsecond shared by the SMs), or what its
// MMAs and their promotion take; plus what a tile costs besides.
bool bsfp8_plan(const Bsfp8Call &c, int (*max_clusters)(int, bool, int), Bsfp8Plan *plan)
{
    const int steps = (c.K + 511) / 512;
    // groups that have any rows (all rows equally likely to fall in each), and the
    // rows of a typical one
    double groups = 1.0;
    if (c.offsets) groups = c.experts * (1.0 - std::pow(1.0 - 1.0 / c.experts, double(c.rows)));
    const double typical = std::max(1.0, c.rows / groups);
    double best = -1;
    const auto consider = [&](int bn, bool pair, int cs) {
        const int per = (steps + cs - 1) / cs;
        if (per * (cs - 1) >= steps) return;  // a slice would be empty
        const int clusters = max_clusters(bn, pair, pair ? 2 : cs);
        if (clusters < 1) return;  // such a cluster does not fit on this GPU
        const double p_tiles = std::ceil(c.N / (pair ? 256.0 : 128.0));
        // (ragged groups end in half a tile on average)
        const double q_tiles = c.offsets && typical > bn ? typical / bn + 0.5 : std::ceil(typical / bn);
        const double rows = std::min(typical / q_tiles, double(bn));
        const double tiles = p_tiles * q_tiles * groups;
        const double bytes = (128 + (pair ? rows / 2 : rows)) * 512;
        const double readers = std::min(tiles, double(clusters)) * (pair ? 2 / q_tiles : cs);
        const double compute = pair ? 1.25 * rows / 256 : bn == 128 ? 1.1 : bn == 64 ? 0.6 : 0.45;
        const double step = std::max({bytes / 100e3, readers * 128 * 512 / 6.3e6, compute});
        const double cost = std::ceil(tiles / clusters) * (per * step + (pair ? 2.5 : 1.0)) + (cs == 1 ? 0.0 : 2.0);
        if (best < 0 || cost < best) {
            best = cost;
            *plan = Bsfp8Plan{bn, pair, cs, 1, groups};
        }
    };
    for (int bn = 16; bn <= 128; bn *= 2) {
        if (bn > 16 && bn >= 2 * typical) break;  // wider than the rows need
        if (typical > 16 * bn) continue;
        for (int cs = 1; cs <= 4; cs *= 2) consider(bn, false, cs);
    }
    if (typical > 64) consider(256, true, 1);
    if (best < 0) consider(128, false, 1);  // (no pairs, and more rows than the loop above takes)
    if (best < 0) return false;
    const int64_t p_tiles = (c.N + (plan->pair ? 255 : 127)) / (plan->pair ? 256 : 128);
    // a group's weights (32 MB of codes) stay in L2 while it runs
    const int64_t slot_bytes = int64_t(plan->pair ? 256 : 128) * bsfp8_code_bytes(c.K);
    plan->group_p = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(p_tiles, (int64_t(32) << 20) / slot_bytes)));
    return true;
}

}  // namespace igemm
