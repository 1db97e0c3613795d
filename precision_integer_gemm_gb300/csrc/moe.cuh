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
