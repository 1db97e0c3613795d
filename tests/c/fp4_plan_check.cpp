// The plan of a 4-bit floating-point product (csrc/fp4_plan.cu, host code) for GPUs on which clusters do not fit.
#include <cstdio>
#include <initializer_list>
#include "fp4.cuh"

using namespace igemm;

static int g_singles, g_clusters, g_pairs;  // CTAs, clusters that split k, pairs that fit

static int fit(int, bool pair, int csize) { return pair ? g_pairs : csize > 1 ? g_clusters : g_singles; }

static int failures;

static void check(bool ok, const char *what, const Fp4Call &c)
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
                for (int rows : {1, 16, 17, 64, 100, 128, 129, 600, 4097, 1 << 20})
                    for (int N : {1, 128, 4096, 28672})
                        for (int K : {1, 512, 4160, 8192, 1 << 20})
                            for (int experts : {0, 1, 5, 64, 1024})
                                for (bool nv : {false, true}) {
                                    g_singles = singles, g_clusters = clusters, g_pairs = pairs;
                                    Fp4Call c{};
                                    c.nv = nv;
                                    c.rows = rows, c.N = N, c.K = K;
                                    c.experts = experts ? experts : 1;
                                    c.offsets = experts ? &some_offsets : nullptr;
                                    Fp4Plan p{};
                                    const bool found = fp4_plan(c, fit, &p);
                                    // a single CTA computes every shape
                                    check(found || singles == 0, "no plan", c);
                                    if (!found) continue;
                                    ++plans;
                                    const int blocks = (K + 511) / 512, per = (blocks + p.cs - 1) / p.cs;
                                    check(fit(p.bn, p.pair, p.cs) > 0, "a cluster that does not fit", c);
                                    check(p.pair ? p.bn == 256 && p.cs == 1 : p.bn >= 16 && p.bn <= 128, "kernel", c);
                                    check(p.cs == 1 || 4 * p.cs <= p.bn, "split", c);
                                    check(per * (p.cs - 1) < blocks, "empty slice", c);
                                    check(p.qt > 0 && p.qt <= p.bn && p.group_p >= 1, "tiles", c);
                                }
    // as many rows as an int holds less the margin that the entry points keep
    g_singles = 152, g_clusters = 36, g_pairs = 76;
    for (int rows : {0x7FFFFFFF - 512, 0x7FFFFFFF - (1 << 22), 0x7FFFFFFF - (1 << 23), 2000000000})
        for (int experts : {0, 1, 7, 1024}) {
            Fp4Call c{};
            c.rows = rows, c.N = 1, c.K = 32;
            c.experts = experts ? experts : 1;
            c.offsets = experts ? &some_offsets : nullptr;
            Fp4Plan p{};
            check(fp4_plan(c, fit, &p) && p.pair && p.qt >= 224 && p.qt <= 256, "most rows", c);
        }
    if (failures) return 1;
    std::printf("fp4 plan ok: %d plans\n", plans);
    return 0;
}
