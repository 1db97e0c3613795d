// Block-scaled fp8 with one float32 scale per 128 k of a row (activations) or per
// 128 rows and 128 k (weights): layout and the calls of its entry points.
#pragma once
#include <atomic>
#include <cstdint>
#include <mutex>
#include <cuda_runtime.h>

namespace igemm {

constexpr int kBsfp8MaxExperts = 1024;
constexpr int kBsfp8MaxTiles = 0x3FFFFFFF;  // of one call

// Bytes of a row of K codes: whole 16-byte units, the tensor maps' row pitch (zero
// codes past K).
constexpr int bsfp8_code_bytes(int K) { return (K / 16 + (K % 16 ? 1 : 0)) * 16; }
// Scales of a row: one per 128 k, rounded up to four (16 bytes).
constexpr int bsfp8_scale_pitch(int K) { return ((K - 1) / 512 + 1) * 4; }

// The answer of ask(), 0 or more, asked for once: `known` keeps one more than it (0: not
// asked yet; no lock once known, a small call asks several times).  Below 0 the question
// failed: 0 this time, and asked again the next.
template <class Ask>
int bsfp8_ask_once(std::atomic<int> &known, std::mutex &mu, Ask ask)
{
    if (const int kept = known.load(std::memory_order_acquire)) return kept - 1;
    std::lock_guard<std::mutex> lock(mu);
    if (!known) {
        const int n = ask();
        if (n < 0) return 0;
        known.store(n + 1, std::memory_order_release);
    }
    return known - 1;
}

// A product: rows x N, dense (offsets null, experts 1) or grouped by expert.
struct Bsfp8Call {
    int format;  // 0 e4m3, 1 e5m2
    const uint8_t *A, *B;
    const float *SFA, *SFB;
    const int *offsets;
    void *C;
    int c_type;
    int rows, experts, N, K;
};

struct Bsfp8Plan {
    int bn;        // most activation rows per tile
    bool pair;     // CTA pairs (256 weight rows)
    int cs;        // CTAs that split k
    int group_p;   // weight tiles per group of the tile order
    double groups;  // expected groups with any rows
    bool stream;   // the weights leave L2 first
};

// The kernel, tile and split for a call; max_clusters(bn, pair, csize) says how
// many clusters of a kernel fit at once (0: none, and the plan does without it).
// False if not even a single CTA fits.
bool bsfp8_plan(const Bsfp8Call &c, int (*max_clusters)(int, bool, int), Bsfp8Plan *plan);
int launch_bsfp8(const Bsfp8Call &c, cudaStream_t stream);

// x [x_rows, K] (element (r, k) at r * ld + k, transposed: at k * ld + r) of type
// x_type, its rows taken in the order of `index` where there is one; a scale per
// tile_rows rows (1 or 128).
struct Bsfp8PackCall {
    int format;
    const void *x;
    int x_type;
    int64_t ld;
    bool transposed;
    const int *index;
    int x_rows;
    int tile_rows;
    uint8_t *codes;
    float *scales;
    int rows, K;
};
int launch_bsfp8_pack(const Bsfp8PackCall &c, cudaStream_t stream);

}  // namespace igemm
