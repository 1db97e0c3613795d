// Routing: what its kernels share, from a block's choices to the sorted pairs.
#pragma once
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "launch.cuh"
#include "ptx.cuh"

namespace igemm {

constexpr int kTB = 64;           // most tokens per block: two mask words
// blocks that one cluster can hold; up to so many do the whole job in one launch
constexpr int kClusterBlocks = 8;
// a block of one cluster takes as many tokens at least (16 x 64 bfloat16, 4 choices: 3.0
// us, 4.2 with 8; 64 x 1024 float32, 8 choices: 11.4 us, 10.7 with 8 and 25.7 with 64)
constexpr int kFewTokens = 16;
constexpr int kRouteThreads = 512;

__device__ __forceinline__ float moe_float(float v) { return v; }
__device__ __forceinline__ float moe_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float moe_float(__half v) { return __half2float(v); }

struct RouteParams {
    const void *logits;
    int *experts;
    float *weights;
    int *offsets, *tokens, *slots;
    int *counts;  // [E][blocks], then exclusive prefixes (three launches)
    int *totals;  // [E]
    uint32_t *packed_counts;  // [blocks][ceil(E / 4)], a byte an expert (two launches)
    int T, E, k, blocks;
    int tb;       // tokens per block
    int normalize;
};

// Order-preserving integer of a logit: larger logits give larger keys, -0 and +0
// the same; NaN counts as -inf, whose key is the lowest.
__device__ __forceinline__ uint32_t route_key(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float route_value(uint32_t key)
{
    return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}
constexpr uint32_t kKeyNone = 0x007FFFFFu;  // of -inf

// Sets in `first[e]` the running sum of `count(e)` over experts below e (warp 0).
template <class F>
__device__ __forceinline__ void route_scan(int *first, int E, F count)
{
    const int lane = threadIdx.x & 31;
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int n = e0 + lane < E ? count(e0 + lane) : 0;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        if (e0 + lane < E) first[e0 + lane] = run + incl - n;
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) first[E] = run;
}

// Places of this block's pairs: first[e] is where its pairs of expert e start.
__device__ __forceinline__ void route_place(const RouteParams &p, const uint2 *mask, const int *first,
                                            const int *experts)
{
    const int t0 = blockIdx.x * p.tb;
    const int n = min(p.tb, p.T - t0) * p.k;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int e = experts[i], t = i / p.k;
        int pos = -1;
        if (e >= 0) {
            const uint2 m = mask[e];
            const uint32_t below = (1u << (t & 31)) - 1u;
            pos = first[e] + (t < 32 ? __popc(m.x & below) : __popc(m.x) + __popc(m.y & below));
            p.tokens[pos] = t0 + t;
        }
        p.slots[static_cast<int64_t>(t0) * p.k + i] = pos;
    }
}

// The block's pairs of each expert (at most kTB) to the launch that places them.
__device__ __forceinline__ void route_counts(const RouteParams &p, const uint2 *mask)
{
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        const int n = __popc(mask[e].x) + __popc(mask[e].y);
        if (p.packed_counts)
            reinterpret_cast<uint8_t *>(p.packed_counts + static_cast<int64_t>(blockIdx.x) * ((p.E + 3) / 4))[e] =
                static_cast<uint8_t>(n);
        else
            p.counts[static_cast<int64_t>(e) * p.blocks + blockIdx.x] = n;
    }
}

// One cluster: from the masks of its blocks to places (THREADS threads a block; first
// [E + 1], start [E] scratch, `chosen` the block's experts).
template <int THREADS>
__device__ __forceinline__ void route_finish(const RouteParams &p, uint2 *mask, int *first, int *start, const int *chosen)
{
    // the pairs of each expert in every block and in those before this one
    const int blocks = gridDim.x;
    if (blocks > 1) cluster_sync_all();
    for (int e = threadIdx.x; e < p.E; e += THREADS) {
        const uint32_t at = smem_u32(mask + e);
        int all = 0, below = 0;
        for (int b = 0; b < blocks; ++b) {
            const uint2 m = blocks > 1 ? ld_cluster_v2(cluster_map(at, b)) : mask[e];
            const int n = __popc(m.x) + __popc(m.y);
            all += n;
            below += b < static_cast<int>(blockIdx.x) ? n : 0;
        }
        first[e] = all;
        start[e] = below;
    }
    __syncthreads();
    if (threadIdx.x < 32) route_scan(first, p.E, [&](int e) { return first[e]; });
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += THREADS) start[e] += first[e];
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= p.E; e += THREADS) p.offsets[e] = first[e];
    for (int i = first[p.E] + blockIdx.x * THREADS + threadIdx.x; i < p.T * p.k; i += blocks * THREADS)
        p.tokens[i] = -1;
    __syncthreads();
    route_place(p, mask, start, chosen);
    if (blocks > 1) cluster_sync_all();  // no block leaves while another may read its masks
}

int launch_route_scan(const RouteParams &p, cudaStream_t stream);
int launch_route_place(const RouteParams &p, int smem, cudaStream_t stream);

// The launches of a routing: choose(p, smem) launches the choice of experts, on the
// blocks of one cluster (p.counts and p.packed_counts null) or on many, of `tb` tokens
// (at most kTB).
template <class Choose>
int route_launch(RouteParams p, cudaStream_t stream, Choose choose, int tb = kTB, int most = kClusterBlocks * kTB)
{
    // up to `most` tokens (512) spread over the blocks of a cluster
    const bool one = p.T <= most;
    p.tb = one ? std::max(kFewTokens, (p.T + kClusterBlocks - 1) / kClusterBlocks) : tb;
    p.blocks = static_cast<int>((int64_t(p.T) + p.tb - 1) / p.tb);
    // the places can sum every block's counts themselves, without a scan, while all of
    // them together read no more than 4 MB (us, two launches and three: 4096 x 256 bfloat16
    // 8.2 and 10.3, 16384 x 64 9.1 and 10.8; 16384 x 256 18.7 and 15.4)
    const int words = (p.E + 3) / 4;
    const bool two = !one && int64_t(p.blocks) * p.blocks * words <= int64_t(1) << 20;
    void *ws = nullptr;
    if (!one) {
        const size_t counts = two ? size_t(words) * p.blocks * 4 : size_t(p.E) * p.blocks * 4;
        if (workspace_alloc(&ws, counts + (two ? 0 : size_t(p.E) * 4), stream) != kOk) return kCudaError;
        if (two) {
            p.packed_counts = static_cast<uint32_t *>(ws);
        } else {
            p.counts = static_cast<int *>(ws);
            p.totals = reinterpret_cast<int *>(static_cast<uint8_t *>(ws) + counts);
        }
    }
    const int smem = p.E * 8 + (p.E + 1) * 4 + p.E * 4 + (one ? kTB * p.k * 4 : 0);
    int rc = choose(p, smem);
    if (rc == kOk && p.counts) rc = launch_route_scan(p, stream);
    if (rc == kOk && !one) rc = launch_route_place(p, smem, stream);
    if (ws && workspace_free(ws, stream) != kOk) rc = kCudaError;
    return rc;
}

}  // namespace igemm
