// Routing of tokens to experts and the weighted sum of the experts' rows.
//
// Routing: a warp per token holds the token's logits in registers (E / 32 per
// lane) as order-preserving integers and takes the largest k times with a warp
// reduction.  The integers of 16-bit logits leave 13 low bits for the expert
// (lower experts count as larger), so one reduction finds value and expert, and up
// to 8 of them are sorted per lane beforehand; float32 logits need a second
// reduction for the lowest expert that holds the value.  A token chooses an expert
// at most once, so the tokens of a block of kTB that chose expert e are one bit
// mask, and a pair's place among its expert's is the number of bits below its
// own: the sort is stable and needs no ordered atomics.  A cluster of up to 8 blocks
// does the whole job for up to 512 tokens, its blocks reading each other's masks in
// shared memory (128 x 256 bfloat16, 8 choices: 5.9 us, where three launches and a
// workspace made a call 4.6 us longer); more tokens take two launches (choice and counts per
// block; places, each block summing the counts of all) or, from some 2^20 words of
// counts read in all, three (a scan over the blocks per expert between them), and
// 16-bit logits of up to 256 experts then go four tokens to a warp
// (moe_choose4_kernel).  Bound by instructions and by the launches: 15.5 us at 16384 x
// 256 bfloat16, 8 choices, whose 10.5 MB are 1.6 us of HBM (alone and cold: choice 13,
// scan 4.5, places 7.5 us).
//
// Combine: bound by HBM, k rows read and one written per token.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include "launch.cuh"
#include "moe.cuh"
#include "moe_route.cuh"
#include "overlap.cuh"
#include "ptx.cuh"

namespace igemm {

constexpr int kChooseThreads = 1024;
constexpr int kChoose4Threads = 32 * kTB / 4;

// The 16-bit form: bits 13 and up of the key, then 0x1FFF - expert.
__device__ __forceinline__ uint32_t route_packed(float v, int e)
{
    return (route_key(v) & ~0x1FFFu) | (0x1FFFu - static_cast<uint32_t>(e));
}
__device__ __forceinline__ float route_packed_value(uint32_t p)
{
    return __uint_as_float((p & 0x80000000u) ? p & 0x7FFFE000u : ~(p | 0x1FFFu));
}

// From every block's counts in bytes: first[e] += all pairs of expert e, start[e] +=
// those of the blocks before this one.  A thread sums four experts over every G-th
// block, as pairs of 16-bit sums (with two launches a thread has at most 64 blocks).
__device__ __forceinline__ void route_sum_counts(const RouteParams &p, int *first, int *start)
{
    const int words = (p.E + 3) / 4, groups = min(kRouteThreads / words, 16);
    const int g = threadIdx.x / words, w = threadIdx.x - g * words;
    if (g >= groups) return;
    const int here = blockIdx.x;
    uint32_t all[2] = {0, 0}, below[2] = {0, 0};  // experts 0 and 2, 1 and 3
#pragma unroll 8
    for (int b = g; b < p.blocks; b += groups) {
        const uint32_t n = p.packed_counts[static_cast<int64_t>(b) * words + w];
        const uint32_t even = n & 0x00FF00FFu, odd = n >> 8 & 0x00FF00FFu;
        all[0] += even;
        all[1] += odd;
        if (b < here) {
            below[0] += even;
            below[1] += odd;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * w + i;
        if (e < p.E) {
            atomicAdd(&first[e], static_cast<int>(all[i & 1] >> (16 * (i >> 1)) & 0xFFFFu));
            atomicAdd(&start[e], static_cast<int>(below[i & 1] >> (16 * (i >> 1)) & 0xFFFFu));
        }
    }
}

// Choice and weights of a block's tokens; their masks; one cluster: everything.
// VPL: logits per lane (E <= 32 VPL); VEC: lane's logits in runs of V (16 bytes at
// most), loaded together.
template <class T, int VPL, bool VEC>
__global__ void __launch_bounds__(kChooseThreads) moe_choose_kernel(const RouteParams p)
{
    constexpr bool kPacked = sizeof(T) == 2;
    constexpr int V = !VEC ? 1 : VPL < 16 / int(sizeof(T)) ? VPL : 16 / int(sizeof(T));
    struct alignas(V * sizeof(T)) Run {
        T v[V];
    };
    extern __shared__ uint2 mask[];  // [E], then (one cluster) first[E + 1], start[E], experts[kTB * k]
    overlap_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool one_cluster = !p.counts && !p.packed_counts;
    int *first = reinterpret_cast<int *>(mask + p.E);
    int *start = first + p.E + 1;
    int *chosen = start + p.E;
    for (int e = threadIdx.x; e < p.E; e += kChooseThreads) mask[e] = make_uint2(0, 0);
    __syncthreads();
    const int t0 = blockIdx.x * p.tb;
    const int mine = min(p.tb, p.T - t0);  // (t0 + tb may pass 2^31)
    for (int i = warp; i < mine; i += kChooseThreads / 32) {
        const int64_t t = t0 + i;
        const T *row = static_cast<const T *>(p.logits) + t * p.E;
        uint32_t key[VPL];  // of expert 32 V (j / V) + V lane + j % V
#pragma unroll
        for (int j = 0; j < VPL; j += V) {
            const int e0 = 32 * j + V * lane;
            Run run;
            if (e0 < p.E) {  // (VEC: E is a multiple of V)
                run = *reinterpret_cast<const Run *>(row + e0);
            } else {
#pragma unroll
                for (int q = 0; q < V; ++q) run.v[q] = T(0.0f);
            }
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float v = moe_float(run.v[q]);
                const uint32_t kk = kPacked ? route_packed(v, e0 + q) : route_key(v);
                key[j + q] = e0 >= p.E ? 0u : v != v ? kKeyNone : kk;
            }
        }
        uint32_t local = 0;  // the lane's largest
        if constexpr (kPacked && VPL <= 8) {
            // sorted: the largest first
#pragma unroll
            for (int r = 0; r < VPL; ++r)
#pragma unroll
                for (int j = r & 1; j + 1 < VPL; j += 2) {
                    const uint32_t a = key[j], b = key[j + 1];
                    key[j] = max(a, b);
                    key[j + 1] = min(a, b);
                }
            local = key[0];
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j) local = max(local, key[j]);
        }
        uint32_t top = __reduce_max_sync(0xffffffffu, local);
        const auto value = [](uint32_t kk) { return kPacked ? route_packed_value(kk) : route_value(kk); };
        const float m = top > kKeyNone ? value(top) : 0.0f;
        float sum = 0.0f;
        if (!p.normalize) {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (key[j] > kKeyNone) sum += expf(value(key[j]) - m);
        }
        // lane c keeps choice c
        int my_e = -1;
        uint32_t my_top = 0;
        for (int c = 0; c < p.k; ++c) {
            if (top <= kKeyNone) break;  // only masked experts are left
            int e;
            bool owner;
            if constexpr (kPacked) {
                owner = local == top;
                e = static_cast<int>(0x1FFFu - (top & 0x1FFFu));
            } else {
                int at = 0x7FFFFFFF;
                if (local == top) {
#pragma unroll
                    for (int j = VPL - 1; j >= 0; --j)
                        if (key[j] == top) at = 32 * (j / V * V) + V * lane + j % V;
                }
                e = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(at)));
                owner = at == e;
            }
            if (lane == c) {
                my_e = e;
                my_top = top;
            }
            if (owner) {  // taken: out of the next rounds
                if constexpr (kPacked && VPL <= 8) {
#pragma unroll
                    for (int j = 0; j + 1 < VPL; ++j) key[j] = key[j + 1];
                    key[VPL - 1] = 0;
                    local = key[0];
                } else {
                    local = 0;
#pragma unroll
                    for (int j = 0; j < VPL; ++j) {
                        if (kPacked ? key[j] == top : 32 * (j / V * V) + V * lane + j % V == e) key[j] = 0u;
                        local = max(local, key[j]);
                    }
                }
            }
            top = __reduce_max_sync(0xffffffffu, local);
        }
        const float my_w = my_e >= 0 ? expf(value(my_top) - m) : 0.0f;
        if (p.normalize) sum = my_w;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane < p.k) {
            p.experts[t * p.k + lane] = my_e;
            p.weights[t * p.k + lane] = my_e >= 0 ? __fdiv_rn(my_w, sum) : 0.0f;
            if (one_cluster) chosen[i * p.k + lane] = my_e;
            if (my_e >= 0) atomicOr(i < 32 ? &mask[my_e].x : &mask[my_e].y, 1u << (i & 31));
        }
    }
    overlap_release();
    __syncthreads();
    if (!one_cluster) {
        route_counts(p, mask);
        return;
    }
    route_finish<kChooseThreads>(p, mask, first, start, chosen);
}

// The larger eight of a descending list and one in ascending places, in descending
// order: elementwise maxima of one against the other reversed hold them as a bitonic
// list, three half-cleaners sort it.
__device__ __forceinline__ void route_merge8(uint32_t (&a)[8], const uint32_t (&b)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = max(a[i], b[7 - i]);
#pragma unroll
    for (int d = 4; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) {
                const uint32_t hi = max(a[i], a[i + d]);
                a[i + d] = min(a[i], a[i + d]);
                a[i] = hi;
            }
}

// The choice of up to 8 among up to 256 experts of 16-bit logits, many tokens: a warp
// takes four tokens at once.  A lane sorts its logits of each token, then lanes merge
// such lists pairwise, halving the tokens that a lane holds (16 lanes apart: two
// tokens each, 8 apart: one), so that eight lanes end with the eight largest of one
// token and lane c of them keeps choice c.  About 400 instructions a token against
// 640 with one token per warp and a reduction per choice (times: launch_choose_vpl).
template <class T, int VPL, bool VEC>
__global__ void __launch_bounds__(kChoose4Threads) moe_choose4_kernel(const RouteParams p)
{
    static_assert(sizeof(T) == 2 && VPL <= 8, "16-bit logits of at most 256 experts");
    constexpr int V = VEC ? VPL : 1;
    struct alignas(V * sizeof(T)) Run {
        T v[V];
    };
    extern __shared__ uint2 mask[];  // [E]
    overlap_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < p.E; e += kChoose4Threads) mask[e] = make_uint2(0, 0);
    __syncthreads();
    const int i0 = 4 * warp;  // within the block
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTB + i0;  // (many tokens: p.tb is kTB)
    Run run[4][VPL / V];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < VPL / V; ++j) {
            const int e0 = 32 * V * j + V * lane;
            if (t0 + q < p.T && e0 < p.E) {  // (VEC: E is a multiple of V)
                run[q][j] = *reinterpret_cast<const Run *>(static_cast<const T *>(p.logits) + (t0 + q) * p.E + e0);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) run[q][j].v[i] = T(-CUDART_INF_F);  // never chosen, adds nothing
            }
        }
    uint32_t list[4][8];  // descending
    float sum[4], top[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            list[q][j] = 0;
            if (j < VPL) {
                const float v = moe_float(run[q][j / V].v[j % V]);
                list[q][j] = v != v ? 0u : route_packed(v, 32 * V * (j / V) + V * lane + j % V);
            }
        }
        const auto order = [&](int a, int b) {
            const uint32_t hi = max(list[q][a], list[q][b]);
            list[q][b] = min(list[q][a], list[q][b]);
            list[q][a] = hi;
        };
        order(0, 1);
        if constexpr (VPL > 2) {
            order(2, 3);
            order(0, 2), order(1, 3);
            order(1, 2);
        }
        if constexpr (VPL > 4) {  // Batcher's odd-even merge of two sorted fours
            order(4, 5), order(6, 7);
            order(4, 6), order(5, 7);
            order(5, 6);
            order(0, 4), order(1, 5), order(2, 6), order(3, 7);
            order(2, 4), order(3, 5);
            order(1, 2), order(3, 4), order(5, 6);
        }
        sum[q] = 0.0f;
        if (!p.normalize) {  // over every expert
            const uint32_t best = __reduce_max_sync(0xffffffffu, list[q][0]);
            top[q] = best > kKeyNone ? route_packed_value(best) : 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const float v = moe_float(run[q][j / V].v[j % V]);
                if (v > -CUDART_INF_F) sum[q] += expf(v - top[q]);  // (not NaN)
            }
        }
    }
    // lanes with bit 4 keep tokens 2 and 3, then those with bit 3 the second of their two
    uint32_t other[8];
#pragma unroll
    for (int n = 2; n; n >>= 1) {
        const bool upper = lane & (8 * n);
#pragma unroll
        for (int q = 0; q < n; ++q) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t give = upper ? list[q][j] : list[q + n][j];
                list[q][j] = upper ? list[q + n][j] : list[q][j];
                other[j] = __shfl_xor_sync(0xffffffffu, give, 8 * n);
            }
            route_merge8(list[q], other);
            const float give = upper ? sum[q] : sum[q + n];
            sum[q] = (upper ? sum[q + n] : sum[q]) + __shfl_xor_sync(0xffffffffu, give, 8 * n);
        }
    }
#pragma unroll
    for (int d = 4; d; d >>= 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) other[j] = __shfl_xor_sync(0xffffffffu, list[0][j], d);
        route_merge8(list[0], other);
        sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], d);
    }
    // (bit 4: the upper two, bit 3: the second of them)
    const int i = i0 + (lane >> 3), c = lane & 7;
    const int64_t t = t0 + (lane >> 3);
    uint32_t mine = list[0][0];
#pragma unroll
    for (int j = 1; j < 8; ++j) mine = c == j ? list[0][j] : mine;
    const int e = c < p.k && mine > kKeyNone ? static_cast<int>(0x1FFFu - (mine & 0x1FFFu)) : -1;
    const float w = e >= 0 ? expf(route_packed_value(mine) - route_packed_value(list[0][0])) : 0.0f;
    float all = w;
#pragma unroll
    for (int d = 4; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    if (!p.normalize) all = sum[0];
    if (t < p.T && c < p.k) {
        p.experts[t * p.k + c] = e;
        p.weights[t * p.k + c] = e >= 0 ? __fdiv_rn(w, all) : 0.0f;
        if (e >= 0) atomicOr(i < 32 ? &mask[e].x : &mask[e].y, 1u << (i & 31));
    }
    overlap_release();
    __syncthreads();
    route_counts(p, mask);
}

// A warp per expert: its counts per block become running sums, 8 blocks a lane.
__global__ void __launch_bounds__(128) moe_scan_kernel(const RouteParams p)
{
    overlap_begin();  // the blocks' counts
    const int e = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= p.E) return;
    int *c = p.counts + static_cast<int64_t>(e) * p.blocks;
    int run = 0;
    for (int b0 = 0; b0 < p.blocks; b0 += 256) {
        int n[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = b0 + 8 * lane + j < p.blocks ? c[b0 + 8 * lane + j] : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += n[j];
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        int at = run + incl - sum;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (b0 + 8 * lane + j < p.blocks) c[b0 + 8 * lane + j] = at;
            at += n[j];
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) p.totals[e] = run;
}

__global__ void __launch_bounds__(kRouteThreads) moe_place_kernel(const RouteParams p)
{
    extern __shared__ uint2 mask[];  // [E], then first[E + 1], start[E]
    int *first = reinterpret_cast<int *>(mask + p.E);
    int *start = first + p.E + 1;
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
        mask[e] = make_uint2(0, 0);
        first[e] = start[e] = 0;
    }
    // the counts; with a scan between, the choices come from the kernel before it,
    // which the scan waited for
    overlap_begin();
    __syncthreads();
    const int t0 = blockIdx.x * p.tb;
    const int n = min(p.tb, p.T - t0) * p.k;
    const int *experts = p.experts + static_cast<int64_t>(t0) * p.k;
    for (int i = threadIdx.x; i < n; i += kRouteThreads) {
        const int e = experts[i], t = i / p.k;
        if (e >= 0) atomicOr(t < 32 ? &mask[e].x : &mask[e].y, 1u << (t & 31));
    }
    if (p.packed_counts) {
        route_sum_counts(p, first, start);
    } else {
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
            first[e] = p.totals[e];
            start[e] = p.counts[static_cast<int64_t>(e) * p.blocks + blockIdx.x];
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) route_scan(first, p.E, [&](int e) { return first[e]; });
    __syncthreads();
    const int64_t pairs = static_cast<int64_t>(p.T) * p.k;
    for (int64_t i = first[p.E] + static_cast<int64_t>(blockIdx.x) * kRouteThreads + threadIdx.x; i < pairs;
         i += static_cast<int64_t>(gridDim.x) * kRouteThreads)
        p.tokens[i] = -1;
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= p.E; e += kRouteThreads) p.offsets[e] = first[e];
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) start[e] += first[e];
    __syncthreads();
    route_place(p, mask, start, experts);
}

template <class T, int VPL>
static int launch_choose_vpl(const RouteParams &p, int smem, cudaStream_t stream)
{
    constexpr int V = VPL < 16 / int(sizeof(T)) ? VPL : 16 / int(sizeof(T));
    const bool vec = p.E % V == 0 && reinterpret_cast<uintptr_t>(p.logits) % (V * sizeof(T)) == 0;
    // 16-bit logits of up to 256 experts, up to 8 choices and more tokens than a cluster's
    // (routing with 8 choices, a token a warp and four: 16384 x 256 bfloat16 20.1 and 15.4
    // us, 65536 x 128 37.5 and 25.5, 8192 x 64 10.4 and 6.6)
    if constexpr (sizeof(T) == 2 && VPL <= 8)
        if (p.T > kClusterBlocks * kTB && p.k <= 8)
            return launch_overlapped(vec ? moe_choose4_kernel<T, VPL, true> : moe_choose4_kernel<T, VPL, false>,
                                     dim3(p.blocks), dim3(kChoose4Threads), smem, stream, p);
    const auto kernel = vec ? moe_choose_kernel<T, VPL, true> : moe_choose_kernel<T, VPL, false>;
    if (p.T > kClusterBlocks * kTB)
        return launch_overlapped(kernel, dim3(p.blocks), dim3(kChooseThreads), smem, stream, p);
    int cluster = 1;
    while (cluster < p.blocks) cluster *= 2;  // (blocks without tokens fill it up)
    return launch_overlapped_clusters(kernel, dim3(cluster), cluster, dim3(kChooseThreads), smem, stream, p);
}

template <class T>
static int launch_choose(const RouteParams &p, int smem, cudaStream_t stream)
{
    if (p.E <= 64) return launch_choose_vpl<T, 2>(p, smem, stream);
    if (p.E <= 128) return launch_choose_vpl<T, 4>(p, smem, stream);
    if (p.E <= 256) return launch_choose_vpl<T, 8>(p, smem, stream);
    if (p.E <= 512) return launch_choose_vpl<T, 16>(p, smem, stream);
    return launch_choose_vpl<T, 32>(p, smem, stream);
}

int launch_route_scan(const RouteParams &p, cudaStream_t stream)
{
    return launch_overlapped(moe_scan_kernel, dim3((p.E + 3) / 4), dim3(128), 0, stream, p);
}
int launch_route_place(const RouteParams &p, int smem, cudaStream_t stream)
{
    return launch_overlapped(moe_place_kernel, dim3(p.blocks), dim3(kRouteThreads), smem, stream, p);
}

int launch_moe_route(const MoeRouteCall &c, cudaStream_t stream)
{
    RouteParams p{};
    p.logits = c.logits;
    p.experts = c.experts;
    p.weights = c.weights;
    p.offsets = c.offsets;
    p.tokens = c.tokens;
    p.slots = c.slots;
    p.T = c.T;
    p.E = c.E;
    p.k = c.k;
    p.normalize = c.normalize ? 1 : 0;
    return route_launch(p, stream, [&](const RouteParams &q, int smem) {
        return c.x_type == 0   ? launch_choose<float>(q, smem, stream)
               : c.x_type == 1 ? launch_choose<__nv_bfloat16>(q, smem, stream)
                               : launch_choose<__half>(q, smem, stream);
    });
}

// ---------------------------------------------------------------- combine
__device__ __forceinline__ void moe_out(float *o, float v) { *o = v; }
__device__ __forceinline__ void moe_out(__nv_bfloat16 *o, float v) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void moe_out(__half *o, float v) { *o = __float2half_rn(v); }

// PER values as one load or store.
template <class T, int PER>
struct alignas(PER * sizeof(T)) MoeRun {
    T v[PER];
};

// A thread per RUNS runs of PER columns of a token, four rows in flight; float32 sums
// in the order of the choices.  Rows of whole 16- or 8-byte runs: one run, threads
// laid over tokens and columns alike (4096 tokens x 8 bfloat16 rows of 4096: 48 us,
// 0.92 of the copy rate).  Other rows: a block of threads per token and 128 RUNS PER
// columns, so that the choices are read once for several narrow loads (rows of 4095:
// 61 us, 147 with a thread per value).  In 8-byte runs that form takes 43 us for rows of
// 4092, where one run takes 49, but 11.9 against 2.5 for rows of 68.  The narrow loads are
// volatile, so all of them go out before the first sum (with plain ones rows of 4095
// took 71 us, of 4094 103 instead of 43, of 4092 59).
template <class T, int PER, int RUNS>
__global__ void __launch_bounds__(128) moe_combine_kernel(const T *Y, const int *slots, const float *weights, T *out, int Tn,
                                                          int k, int N)
{
    using Run = MoeRun<T, PER>;
    overlap_wait();
    int64_t t;
    uint32_t n;  // (unsigned: a row's last threads may lie past 2^31)
    if constexpr (RUNS == 1) {
        const uint32_t per_row = static_cast<uint32_t>(N / PER);
        const uint64_t item = static_cast<uint64_t>(blockIdx.x) * 128 + threadIdx.x;
        t = static_cast<int64_t>(item / per_row);
        if (t >= Tn) return;
        n = static_cast<uint32_t>(item - static_cast<uint64_t>(t) * per_row) * PER;
    } else {
        const uint32_t chunks = (static_cast<uint32_t>(N) + 128 * RUNS * PER - 1) / (128 * RUNS * PER);
        t = blockIdx.x / chunks;
        n = (blockIdx.x - static_cast<uint32_t>(t) * chunks) * (128 * RUNS * PER) + threadIdx.x * PER;
    }
    const int64_t rows = static_cast<int64_t>(Tn) * k;
    const uint32_t width = static_cast<uint32_t>(N);
    float acc[RUNS][PER];
#pragma unroll
    for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[r][i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 4) {
        Run v[4][RUNS];
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = t * k + j0 + j;
            const int64_t s = j0 + j < k ? slots[at] : -1;
            const bool live = s >= 0 && s < rows;
            w[j] = live ? weights[at] : 0.0f;
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
#pragma unroll
                for (int i = 0; i < PER; ++i) v[j][r].v[i] = T(0.0f);
                const uint32_t nr = n + r * (128 * PER);
                if (live && nr < width) {
                    const T *from = Y + s * N + nr;
                    if constexpr (sizeof(Run) == 16)
                        *reinterpret_cast<uint4 *>(&v[j][r]) = ld_stream_v4(from);
                    else
                        ld_once(v[j][r], from);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < RUNS; ++r)
#pragma unroll
                for (int i = 0; i < PER; ++i) acc[r][i] = fmaf(w[j], moe_float(v[j][r].v[i]), acc[r][i]);
    }
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
        const uint32_t nr = n + r * (128 * PER);
        if (nr >= width) break;
        Run o;
#pragma unroll
        for (int i = 0; i < PER; ++i) moe_out(&o.v[i], acc[r][i]);
        *reinterpret_cast<Run *>(out + t * N + nr) = o;
    }
    overlap_release();
}

template <class T, int PER>
static int launch_combine_per(const MoeCombineCall &c, cudaStream_t stream)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(c.Y) | reinterpret_cast<uintptr_t>(c.out);
    if constexpr (PER > 1)
        if (at % (PER * sizeof(T)) != 0 || c.N % PER != 0) return launch_combine_per<T, PER / 2>(c, stream);
    constexpr int kRuns = PER * sizeof(T) >= 8 ? 1 : 4;
    const int64_t chunk = int64_t(128) * kRuns * PER;
    const int64_t blocks = kRuns == 1 ? (int64_t(c.T) * (c.N / PER) + 127) / 128 : c.T * ((c.N + chunk - 1) / chunk);
    if (blocks > 0x7FFFFFFF) return kUnsupportedShape;
    return launch_overlapped(moe_combine_kernel<T, PER, kRuns>, dim3(static_cast<unsigned>(blocks)), dim3(128), 0,
                             stream, static_cast<const T *>(c.Y), c.slots, c.weights, static_cast<T *>(c.out), c.T, c.k,
                             c.N);
}

int launch_moe_combine(const MoeCombineCall &c, cudaStream_t stream)
{
    switch (c.x_type) {
    case 0: return launch_combine_per<float, 4>(c, stream);
    case 1: return launch_combine_per<__nv_bfloat16, 8>(c, stream);
    default: return launch_combine_per<__half, 8>(c, stream);
    }
}

}  // namespace igemm
