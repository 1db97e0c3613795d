// What a block-scaled fp8 product asks about its kernels (csrc/bsfp8.cuh) is asked once, also where the answer is
// that a kernel cannot run; a question that failed is asked again.
#include <cstdio>
#include <initializer_list>
#include "bsfp8.cuh"

using namespace igemm;

static int failures;

static void check(bool ok, const char *what, int answer)
{
    if (ok) return;
    ++failures;
    std::printf("%s: %d\n", what, answer);
}

int main()
{
    for (int answer : {0, 1, 76, 152}) {
        std::atomic<int> known{0};
        std::mutex mu;
        int asked = 0;
        const auto ask = [&] {
            ++asked;
            return asked == 1 ? -1 : answer;
        };
        check(bsfp8_ask_once(known, mu, ask) == 0, "a question that failed", answer);
        for (int i = 0; i < 5; ++i) check(bsfp8_ask_once(known, mu, ask) == answer, "the answer", answer);
        check(asked == 2, "times asked", asked);
    }
    if (failures) return 1;
    std::printf("ask once ok\n");
    return 0;
}
