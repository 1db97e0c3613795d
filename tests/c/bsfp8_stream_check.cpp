// Which block-scaled fp8 products mark their weights as the first to leave L2 (csrc/bsfp8_plan.cu, host code): large ones
// that are read once, not those that most groups read again.
#include <cstdio>
#include "bsfp8.cuh"

using namespace igemm;

static int fit(int, bool pair, int csize) { return pair ? 76 : csize == 1 ? 152 : csize == 2 ? 76 : 36; }

static int failures;

static void check(int rows, int N, int K, int experts, bool want)
{
    static const int some_offsets = 0;
    Bsfp8Call c{};
    c.rows = rows, c.N = N, c.K = K, c.c_type = 1;
    c.experts = experts ? experts : 1;
    c.offsets = experts ? &some_offsets : nullptr;
    c.C = reinterpret_cast<void *>(uintptr_t(0x10000));
    Bsfp8Plan p{};
    if (bsfp8_plan(c, fit, &p) && p.stream == want && !(p.stream && p.pair)) return;
    ++failures;
    std::printf("rows %d N %d K %d experts %d: kernel of %d%s, stream %d\n", rows, N, K, experts, p.bn, p.pair ? " (pair)" : "",
                p.stream);
}

int main()
{
    check(16, 28672, 8192, 0, true);
    check(128, 28672, 8192, 0, true);
    check(16, 4096, 4096, 0, false);     // 16 MB
    check(8192, 8192, 8192, 0, false);   // pairs
    check(32, 4096, 4096, 64, true);
    check(512, 4096, 4096, 64, true);
    check(2048, 4096, 4096, 64, true);
    check(4096, 4096, 4096, 64, false);  // half of the groups have more than the tile's 64 rows
    check(8192, 4096, 4096, 64, false);
    check(8192, 4096, 4096, 128, false);
    check(32768, 4096, 4096, 64, false);
    if (failures) return 1;
    std::printf("bsfp8 stream ok\n");
    return 0;
}
