// Host only: the kernel, tile and split of a block-scaled fp8 product.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include "bsfp8.cuh"

namespace igemm {

// Kernel, tile and split by estimated time in microseconds: 4.5 for the start, then every
// wave of tiles its groups of 512 k and what a tile costs besides.  A group takes an SM
// 0.83 with tiles of 16 activations, 0.86 with 32, 0.92 with 64, 1.55 with 128, a CTA pair
// 1.6 (up to 128) or 1.75, or what HBM takes to bring the weights of all SMs at work, 6.3 MB
// a microsecond.  A split of k over two or four CTAs adds up to 2.7, with 64 activations
// or more to every wave (7 with 128).  (4096 x 4096 weights and 16 activations: 11.3 whole,
// 8.7 on two, 8.3 on four; 64: 12.1, 10.7, 9.9; 128 activations as two tiles of 64: 12.3,
// as one 16.0; 8192 x 8192: 256 activations as two tiles of 128 28, on pairs 34.7; 768: 76
// and 68.)
bool bsfp8_plan(const Bsfp8Call &c, int (*max_clusters)(int, bool, int), Bsfp8Plan *plan)
{
    const int steps = (c.K + 511) / 512;
    // groups that have any rows (all rows equally likely to fall in each), and the
    // rows of a typical one
    double groups = 1.0;
    if (c.offsets) groups = c.experts * (1.0 - std::pow(1.0 - 1.0 / c.experts, double(c.rows)));
    const double typical = std::max(1.0, c.rows / groups);
    // where rows of C start
    const uintptr_t rows_at = reinterpret_cast<uintptr_t>(c.C) | uintptr_t(c.N) * (c.c_type == 0 ? 4 : 2);
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
        const double compute = pair ? (rows <= 128 ? 1.6 : 1.75) : bn == 128 ? 1.55 : bn == 64 ? 0.92 : bn == 32 ? 0.86 : 0.83;
        const double split = cs == 1 ? 0.0 : bn == 128 ? 7.0 : bn == 64 ? 2.1 + 0.15 * cs : bn == 32 ? 1.8 + 0.2 * cs : 0.4 + 0.1 * cs;
        // (pairs: a lane's row of C, straight from registers or through shared memory)
        const double tile = pair        ? 2.4 + (c.c_type == 0 ? 0.6 : 0.0) + (rows_at % 32 == 0 ? 0.0 : 0.8)
                            : bn == 128 ? (c.c_type == 0 ? 1.5 : 0.8)
                                        : 0.5;
        // a wave of n clusters: they read the weights of n / q_tiles tiles
        const auto wave = [&](double n) {
            const double weights = n * (pair ? 2 : cs) / std::min(q_tiles, n) * 128 * 512;
            return per * std::max(compute, weights / 6.3e6) + tile + (bn >= 64 ? split : 0.0);
        };
        const double full = std::floor(tiles / clusters), rest = tiles - full * clusters;
        const double cost = full * wave(clusters) + (rest > 0.01 ? wave(rest) : 0.0) + (bn >= 64 ? 0.0 : split);
        if (best < 0 || cost < best) {
            best = cost;
            *plan = Bsfp8Plan{bn, pair, cs, 1, groups, false};
        }
    };
    for (int bn = 16; bn <= 128; bn *= 2) {
        if (bn > 16 && bn >= 2 * typical) break;  // wider than the rows need
        if (typical > 16 * bn) continue;
        for (int cs = 1; cs <= 4; cs *= 2) consider(bn, false, cs);
    }
    // (Not with rows of C that only 2-byte pieces reach, a lane a row.  What that costs 16-bit C of
    // odd N, N = 8191 and 8190, K = 8192, us: 600 rows 80 and 61, 2048 186 and 120, 4096 369 and 207;
    // float32 C of odd N stays on pairs, 226 at 4096.)
    if (typical > 64 && rows_at % 4 == 0) consider(256, true, 1);
    if (best < 0) consider(128, false, 1);  // (no pairs, and more rows than the loop above takes)
    if (best < 0) return false;
    const int64_t p_tiles = (c.N + (plan->pair ? 255 : 127)) / (plan->pair ? 256 : 128);
    // a group's weights (32 MB of codes) stay in L2 while it runs
    const int64_t slot_bytes = int64_t(plan->pair ? 256 : 128) * bsfp8_code_bytes(c.K);
    plan->group_p = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(p_tiles, (int64_t(32) << 20) / slot_bytes)));
    // Weights from 24 MB on leave L2 first, before what other kernels left there (us, with and
    // without: 64 x 28672 x 8192 42.4 and 43.3, two tiles of 64 50.9 and 51.7; 512 rows over 64
    // experts of 4096 x 4096 157.3 and 158.5), but where many groups of several have more rows than
    // a tile and read theirs again (4096 rows over 64 experts 196 and 184, 3600 over 128 359 and
    // 328, 8192 389 and 362; with fewer rows a group than two thirds of a tile within 1 %).
    plan->stream = !plan->pair && groups * c.N * double(bsfp8_code_bytes(c.K)) >= 24.0 * (1 << 20) &&
                   (!c.offsets || 3 * typical <= 2 * plan->bn);
    return true;
}

}  // namespace igemm
