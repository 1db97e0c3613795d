// The 4-bit floating-point formats' layout and the calls of their entry points.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace igemm {

// Bytes of a row of K packed e2m1 codes: whole blocks of 32 (zero codes past K).
constexpr int fp4_code_bytes(int K) { return (K / 32 + (K % 32 ? 1 : 0)) * 16; }
// Bytes from one row's scales to the next: one byte per block of 32 k (mx) or 16
// k (nv), rounded up to 16 (the tensor maps' row pitch).
constexpr int fp4_scale_pitch(int K, bool nv) { return ((K - 1) / (nv ? 256 : 512) + 1) * 16; }

// A product: rows x N, dense (offsets null, experts 1) or grouped by expert.
struct Fp4Call {
    bool nv;
    const uint8_t *A, *B, *SFA, *SFB;
    const int *offsets;
    const float *alpha;
    void *C;
    int c_type;
    int rows, experts, N, K;
};

struct Fp4Plan {
    int bn;        // most activation rows per tile
    bool pair;     // CTA pairs (256 weight rows)
    int cs;        // CTAs that split k
    int qt;        // activation rows per tile
    int group_p;   // weight tiles per group of the tile order
    double groups;  // expected groups with any rows
};

// The kernel, tile and split for a call; max_clusters(bn, pair, csize) says how
// many clusters of a kernel fit at once (0: none, and the plan does without it).
// False if not even a single CTA fits.
bool fp4_plan(const Fp4Call &c, int (*max_clusters)(int, bool, int), Fp4Plan *plan);

int launch_fp4_mx(const Fp4Call &c, cudaStream_t stream);
int launch_fp4_nv(const Fp4Call &c, cudaStream_t stream);

// x [x_rows, K] (element (r, k) at r * ld + k, transposed: at k * ld + r) of type
// x_type, its rows taken in the order of `index` where there is one.
struct Fp4PackCall {
    bool nv;
    const void *x;
    int x_type;
    int64_t ld;
    bool transposed;
    const int *index;
    int x_rows;
    const float *tensor_scale;
    uint8_t *codes, *scales;
    int rows, K;
};
int launch_fp4_pack(const Fp4PackCall &c, cudaStream_t stream);

}  // namespace igemm
