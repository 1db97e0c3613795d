// Host only: the kernel, tile and split of a 4-bit floating-point product.
#include <algorithm>
#include <cmath>
#include "fp4.cuh"

namespace igemm {

// Kernel, tile and split by estimated time in microseconds.  A wave of tiles takes
// blocks of 512 k times the time to bring a block to an SM, 90 KB a microsecond
// from L2 (64 KB to 70 KB for 0.72 us in 128 x 128 and 256 x 256 tiles, 36 KB for 0.37
// us in 128 x 16), or HBM's 6.3 MB a microsecond shared by the SMs (on CTA pairs:
// those that read different weights), plus what a tile costs besides (1 us; 3.2 us
// on CTA pairs).
// A split of k adds 2 us (4 us for 64 activation rows: 64 x 8192 x 8192 12.0 us
// split, 10.3 whole; with 128 it never paid).
// Against the fastest of all choices on 90 shapes (activations 1 .. 2048, weights
// 128 x 65536 .. 28672 x 8192) the choice is within 3 % on 79, within 12 % on 85, and
// 16 to 22 % behind on five: a single token through 4096 x 4096 that two CTAs should
// split, 40 and 64 rows through 28672 x 8192 that nobody should, 200 x 4096 x 14336
// and 2048 x 128 x 65536 that do not belong on CTA pairs.
bool fp4_plan(const Fp4Call &c, int (*max_clusters)(int, bool, int), Fp4Plan *plan)
{
    const int blocks = (c.K + 511) / 512;
    // groups that have any rows (all rows equally likely to fall in each), and the
    // rows of a typical one
    double groups = 1.0;
    if (c.offsets) groups = c.experts * (1.0 - std::pow(1.0 - 1.0 / c.experts, double(c.rows)));
    const double typical = std::max(1.0, c.rows / groups);
    const double scale_bytes = c.nv ? 32.0 : 16.0;
    double best = -1;
    const auto consider = [&](int bn, bool pair, int cs, int qt) {
        const int per = (blocks + cs - 1) / cs;
        if (per * (cs - 1) >= blocks) return;  // a slice would be empty
        const int clusters = max_clusters(bn, pair, pair ? 2 : cs);
        if (clusters < 1) return;  // such a cluster does not fit on this GPU
        const double p_tiles = std::ceil(c.N / (pair ? 256.0 : 128.0));
        // (ragged groups end in half a tile on average)
        const double q_tiles = c.offsets && typical > bn ? typical / bn + 0.5 : std::ceil(typical / qt);
        const double rows = std::min(typical / q_tiles, double(qt));
        const double tiles = p_tiles * q_tiles * groups;
        const double bytes = (128 + (pair ? rows / 2 : rows)) * 256 + (128 + rows) * scale_bytes;
        const double readers = std::min(tiles, double(clusters)) * (pair ? 2 / q_tiles : cs);
        const double block = std::max(bytes / 90e3, readers * 128 * (256 + scale_bytes) / 6.3e6);
        const double cost = std::ceil(tiles / clusters) * (per * block + (pair ? 3.2 : 1.0)) +
                            (cs == 1 ? 0.0 : bn == 64 ? 4.0 : 2.0);
        if (best < 0 || cost < best) {
            best = cost;
            *plan = Fp4Plan{bn, pair, cs, qt, 1, groups};
        }
    };
    for (int bn = 16; bn <= 128; bn *= 2) {
        if (bn > 16 && bn >= 2 * typical) break;  // wider than the rows need
        if (typical > 16 * bn) continue;
        for (int cs = 1; cs <= (bn == 128 ? 1 : bn == 16 ? 4 : 8); cs *= 2)
            consider(bn, false, cs, bn);
    }
    if (typical > 128) {
        // one group: as many equal tiles as fill the last wave best
        const int64_t least = c.offsets ? 1 : (int64_t(c.rows) + 255) / 256;
        for (int64_t n = least; n <= (c.offsets ? 1 : least + 2); ++n)
            consider(256, true, 1,
                     c.offsets ? 256 : static_cast<int>(std::min<int64_t>(256, ((c.rows + n - 1) / n + 31) / 32 * 32)));
    }
    if (best < 0) consider(128, false, 1, 128);  // (no pairs, and more rows than the loop above takes)
    if (best < 0) return false;
    const int64_t p_tiles = (c.N + (plan->pair ? 255 : 127)) / (plan->pair ? 256 : 128);
    // a group's weights (32 MB of codes) stay in L2 while it runs
    const int64_t slot_bytes = int64_t(plan->pair ? 256 : 128) * fp4_code_bytes(c.K);
    plan->group_p = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(p_tiles, (int64_t(32) << 20) / slot_bytes)));
    return true;
}

}  // namespace igemm
