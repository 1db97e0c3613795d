// The plan of a block-scaled fp8 product (csrc/bsfp8_plan.cu, host code) for GPUs on which clusters do not fit.
#include <cstdio>
#include <initializer_list>
#include "bsfp8.cuh"

using namespace igemm;

static int g_singles, g_clusters, g_pairs;  // CTAs, clusters that split k, pairs that fit

static int fit(int, bool pair, int csize) { return pair ? g_pairs : csize > 1 ? g_clusters : g_singles; }

static int failures;

static void check(bool ok, const char *what, const Bsfp8Call &c)
{
    if (ok) return;
    ++failures;
    std::printf("%s: rows %d N %d K %d experts %d, singles %d clusters %d pairs %d\n", what, c.rows, c.N, c.K, c.experts,
                g_singles, g_clusters, g_pairs);
}

int main()
{
    static const int some_offsets = 0;
    int plans = 0;
    for (int singles : {152, 1, 0})
        for (int clusters : {36, 0})
            for (int pairs : {76, 0})
                for (int rows : {1, 16, 17, 64, 100, 128, 129, 600, 4097, 1 << 20, 0x7FFFFFFF - 512})
                    for (int N : {1, 129, 4096, 28672})
                        for (int K : {1, 512, 4160, 8192, 1 << 22})
                            for (int experts : {0, 1, 5, 64, 1024})
                                for (int c_type : {0, 1})
                                    for (uintptr_t at : {uintptr_t(0x10000), uintptr_t(0x10002)}) {
                                        if (c_type == 0 && at % 4) continue;
                                        g_singles = singles, g_clusters = clusters, g_pairs = pairs;
                                        Bsfp8Call c{};
                                        c.rows = rows, c.N = N, c.K = K;
                                        c.experts = experts ? experts : 1;
                                        c.offsets = experts ? &some_offsets : nullptr;
                                        c.C = reinterpret_cast<void *>(at);
                                        c.c_type = c_type;
                                        Bsfp8Plan p{};
                                        const bool found = bsfp8_plan(c, fit, &p);
                                        // a single CTA computes every shape
                                        check(found || singles == 0, "no plan", c);
                                        if (!found) continue;
                                        ++plans;
                                        const int steps = (K + 511) / 512, per = (steps + p.cs - 1) / p.cs;
                                        check(fit(p.bn, p.pair, p.cs) > 0, "a cluster that does not fit", c);
                                        check(p.pair ? p.bn == 256 && p.cs == 1
                                                     : p.bn == 16 || p.bn == 32 || p.bn == 64 || p.bn == 128,
                                              "kernel", c);
                                        check(p.cs == 1 || p.cs == 2 || p.cs == 4, "split", c);
                                        check(per * (p.cs - 1) < steps, "empty slice", c);
                                        check(p.group_p >= 1 && p.groups > 0 && p.groups <= c.experts, "tiles", c);
                                        // pairs store rows of C in words
                                        check(!p.pair || c_type == 0 || (N % 2 == 0 && at % 4 == 0), "rows of C", c);
                                    }
    if (failures) return 1;
    std::printf("bsfp8 plan ok: %d plans\n", plans);
    return 0;
}
