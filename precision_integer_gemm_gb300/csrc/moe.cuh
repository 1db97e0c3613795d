// The row passes around the products grouped by expert.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace igemm {

struct MoeRouteCall {
    const void *logits;  // [T, E] of type x_type
    int x_type;          // 0 float32, 1 bfloat16, 2 float16
    int *experts;        // [T, k]
    float *weights;      // [T, k]
    int *offsets;        // [E + 1]
    int *tokens;         // [T * k]
    int *slots;          // [T, k]
    int T, E, k;
    bool normalize;
};
int launch_moe_route(const MoeRouteCall &c, cudaStream_t stream);

// Routing by scores: softmax or sigmoid, a bias for the choice, groups of experts.
struct MoeScoredCall {
    MoeRouteCall route;
    const float *bias;  // [E] or null
    int score;          // 0 softmax, 1 sigmoid
    int groups, group_k, group_top;
    float scale;
};
int launch_moe_route_scored(const MoeScoredCall &c, cudaStream_t stream);

// Gradient of the logits [T, E] for that of the weights.
struct MoeScoredGradCall {
    const void *logits;
    int x_type;
    const int *experts;     // [T, k]
    const float *dweights;  // [T, k]
    void *dlogits;          // [T, E] of type x_type
    int T, E, k, score;
    bool normalize;
    float scale;
};
int launch_moe_route_scored_grad(const MoeScoredGradCall &c, cudaStream_t stream);

struct MoeCombineCall {
    const void *Y;  // [T * k, N] of type x_type
    int x_type;
    const int *slots;
    const float *weights;
    void *out;      // [T, N] of type x_type
    int T, k, N;
};
int launch_moe_combine(const MoeCombineCall &c, cudaStream_t stream);

}  // namespace igemm
