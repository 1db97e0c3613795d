// Routing by scores and its gradient.
//
//   s = softmax(x) or 1 / (1 + e^-x) over the E experts of a token, c = s + bias; a group's
//   score is the sum of its one or two largest c; the choice is the k largest c among the
//   experts of the best groups, the weight scale * s, over the sum of the chosen s where
//   they are renormalised.
//
// The choice is that of the definition in 64 bits, ties to the lowest expert: a token's c
// are computed in 32 bits, and where two that decide are nearer than the rounding could
// be, these alone are computed again, a lane each: neighbours among the chosen and those
// left behind the last of them (some tokens in a thousand), the largest experts of groups
// at the border between taken and left (one token in ten thousand).  (The 64-bit pipe is
// slow: a token's 256 scores take a warp 40 us, one a lane 2.)  A token with more of them
// than a warp has lanes is done again as a whole, after the block's others.  Without a bias
// (none given, or zeros, as before the first step of a training) the scores are in the order
// of the logits, which are compared as they are; a group's two largest then are those of its
// logits, and scores are told apart by their relative error.
//
// A warp per token, a lane E / 32 neighbouring experts, so that a group is a run of lanes
// and the first lane with the largest value holds the lowest expert.  From the choices to
// the sorted pairs everything is as without scores (moe_route.cuh).
//
// The k largest: the k-th largest of the lanes' largest bounds the k-th largest of all from
// below, so the few experts not below it go to a list, one a lane, and are ranked there (one
// maximum after another, a lane's next looked for in turn: 37.1 us where this takes 32.1).
// The weights come last, several tokens a warp (29.2 us).
//
// Bound by instructions: 16384 x 256 float32, 8 choices, by sigmoid 20.4 us without bias or
// groups, 24.7 with a bias, 29.5 with 8 groups by their two best as well (1057 warp
// instructions a token, issue slots 67 % busy; reading the logits is 2.5 us).
#include <algorithm>
#include <math_constants.h>
#include "launch.cuh"
#include "moe.cuh"
#include "moe_route.cuh"
#include "overlap.cuh"
#include "ptx.cuh"

namespace igemm {

constexpr int kScoredThreads = 512;

struct ScoredParams {
    RouteParams r;
    const float *bias;
    int sigmoid;
    int groups, per, group_k, two;  // per: experts of a group; two: its two largest count
    float scale;
    int vec;  // rows of whole runs
};

// (Below -88 it is e^x to every bit, down to the smallest float32; e^-x passes the largest at 88.7.)
__device__ __forceinline__ float scored_sigmoid(float x)
{
    return x < -88.0f ? expf(x) : __fdiv_rn(1.0f, 1.0f + expf(-x));
}
// For the choice: within 1.63 2^-22 (an exponential of 2 + 1.173 |x| ulp counts s (1 - s),
// the sum 2^-24, the quotient 2 ulp).
__device__ __forceinline__ float scored_sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// Order-preserving integers of 64-bit scores (comparisons of doubles are as slow as their sums).
__device__ __forceinline__ uint64_t scored_key(double v)
{
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ double scored_value(uint64_t k)
{
    return __longlong_as_double(static_cast<long long>(k >> 63 ? k & ~(uint64_t(1) << 63) : ~k));
}
constexpr uint64_t kKey64None = 0x000FFFFFFFFFFFFFull;  // of -inf

// The logit as it counts: NaN is -inf.
template <class T>
__device__ __forceinline__ float scored_logit(const T *row, int e)
{
    const float v = moe_float(row[e]);
    return v != v ? -CUDART_INF_F : v;
}

// a1 >= a2: the two largest so far; v another.
template <class F>
__device__ __forceinline__ void scored_two(F &a1, F &a2, F v)
{
    a2 = v > a1 ? a1 : v > a2 ? v : a2;
    a1 = v > a1 ? v : a1;
}

__device__ __forceinline__ void scored_two(float &a1, float &a2, float v)
{
    a2 = fmaxf(a2, fminf(a1, v));
    a1 = fmaxf(a1, v);
}
// ... and two others, b1 >= b2.
__device__ __forceinline__ void scored_join(float &a1, float &a2, float b1, float b2)
{
    a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
    a1 = fmaxf(a1, b1);
}

// The sum of a group's largest, or of its two largest where there are two.  (Sums past the range
// stay at its end: -inf is a group of no experts, and the bounds of such sums are infinite, so that
// 64 bits decide.)
__device__ __forceinline__ float scored_group(float a1, float a2, bool two)
{
    if (!two || !(a2 > -CUDART_INF_F)) return a1;
    return fmaxf(fminf(a1 + a2, CUDART_MAX_NORMAL_F), -CUDART_MAX_NORMAL_F);
}

// How far a group's score may be off its value: twice the error of a c's score (`slack`), and
// relative to the sizes of its parts, which a sum of both signs does not show, the roundings of
// the two c (2^-24 each of its own), of their sum and of the bounds that the score is compared by.
// Without a bias the parts are positive and within 143 2^-23 (e^-y, y up to 84), or below 2^-120.
__device__ __forceinline__ float scored_slip(float a1, float a2, bool two, float slack, bool biased)
{
    const float size = fabsf(a1) + (two && a2 > -CUDART_INF_F ? fabsf(a2) : 0.0f);
    const float slip = slack + 0x1p-22f * size;
    return biased ? slip : fminf(slip, 0x1p-15f * size + 0x1p-120f);
}

// Bit g: group g is taken; lane g holds its score (`none`: nothing to choose).
template <class F>
__device__ __forceinline__ uint32_t scored_groups(F score, F none, int groups, int group_k)
{
    const int lane = threadIdx.x & 31;
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
        const F other = __shfl_sync(0xffffffffu, score, g);
        rank += other > score || (other == score && g < lane) ? 1 : 0;
    }
    return __ballot_sync(0xffffffffu, lane < groups && rank < group_k && score > none);
}

// One expert's c in 64 bits; softmax: with the row's largest logit and sum.
__device__ __forceinline__ double scored_c_64(const ScoredParams &p, double x, int e, double m, double sum)
{
    const double s = p.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / sum;
    return p.bias ? s + static_cast<double>(p.bias[e]) : s;
}

// A softmax row's sum in 64 bits (m: its largest logit).
template <class T, int VPL>
__device__ __noinline__ double scored_sum_64(const ScoredParams &p, const T *row, float m)
{
    const int e0 = (threadIdx.x & 31) * VPL;
    double sum = 0.0;
#pragma unroll 4
    for (int j = 0; j < VPL; ++j)
        if (e0 + j < p.r.E) sum += exp(static_cast<double>(scored_logit(row, e0 + j)) - static_cast<double>(m));
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum;
}

// The whole choice in 64 bits: lane i's expert, -1 where none is left.
template <class T, int VPL>
__device__ __noinline__ int scored_choose_64(const ScoredParams &p, const T *row, bool biased)
{
    const int lane = threadIdx.x & 31, e0 = lane * VPL;
    uint64_t c[VPL], s[VPL];  // what experts and groups are chosen by
    float m = -CUDART_INF_F;
    for (int j = 0; j < VPL; ++j)
        if (e0 + j < p.r.E) m = fmaxf(m, scored_logit(row, e0 + j));
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const double sum = p.sigmoid ? 1.0 : scored_sum_64<T, VPL>(p, row, m);
    for (int j = 0; j < VPL; ++j) {
        const float x = e0 + j < p.r.E ? scored_logit(row, e0 + j) : -CUDART_INF_F;
        c[j] = s[j] = kKey64None;
        if (x > -CUDART_INF_F) {
            const double v = scored_c_64(p, x, e0 + j, m, sum);
            const uint64_t k = v == v ? scored_key(v) : kKey64None;
            c[j] = biased ? k : scored_key(x);
            s[j] = biased || p.two ? k : c[j];
        }
    }
    if (p.groups > 1) {
        uint64_t score = kKey64None;
        for (int g = 0; g < p.groups; ++g) {
            uint64_t a1 = kKey64None, a2 = kKey64None;
            for (int j = 0; j < VPL; ++j)
                if (c[j] > kKey64None && (e0 + j) / p.per == g) scored_two(a1, a2, s[j]);
            for (int d = 16; d; d >>= 1) {
                const uint64_t b1 = __shfl_xor_sync(0xffffffffu, a1, d), b2 = __shfl_xor_sync(0xffffffffu, a2, d);
                scored_two(a1, a2, b1);
                scored_two(a1, a2, b2);
            }
            if (lane == g)
                score = p.two && a2 > kKey64None ? scored_key(scored_value(a1) + scored_value(a2)) : a1;
        }
        const uint32_t taken = scored_groups(score, kKey64None, p.groups, p.group_k);
        for (int j = 0; j < VPL; ++j)
            if (e0 + j < p.r.E && !(taken >> ((e0 + j) / p.per) & 1u)) c[j] = kKey64None;
    }
    int mine = -1;
    for (int i = 0; i < p.r.k; ++i) {
        uint64_t best = kKey64None;
        int e = 0x7FFFFFFF;
        for (int j = 0; j < VPL; ++j)
            if (c[j] > best) {
                best = c[j];
                e = e0 + j;
            }
        for (int d = 16; d; d >>= 1) {
            const uint64_t b = __shfl_xor_sync(0xffffffffu, best, d);
            const int f = __shfl_xor_sync(0xffffffffu, e, d);
            if (b > best || (b == best && f < e)) {
                best = b;
                e = f;
            }
        }
        if (best <= kKey64None) break;
        if (lane == i) mine = e;
        for (int j = 0; j < VPL; ++j)
            if (e0 + j == e) c[j] = kKey64None;
    }
    return mine;
}

// The first n lanes hold experts by falling c in 32 bits, among them every one that could
// be among the k largest; the same by c in 64 bits, lanes from k on -1.
__device__ __forceinline__ int scored_order_64(const ScoredParams &p, int e, float x, int n, double m, double sum)
{
    const int lane = threadIdx.x & 31;
    const uint64_t key = lane < n ? scored_key(scored_c_64(p, x, e, m, sum)) : kKey64None;
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const uint64_t other = __shfl_sync(0xffffffffu, key, i);
        const int f = __shfl_sync(0xffffffffu, e, i);
        rank += other > key || (other == key && f < e) ? 1 : 0;
    }
    int mine = -1;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const int r = __shfl_sync(0xffffffffu, rank, i), f = __shfl_sync(0xffffffffu, e, i);
        if (r == lane && lane < p.r.k) mine = f;
    }
    return mine;
}

// The groups of `border` may be taken or not: bit j of a lane's `cand` says that its expert j
// may count in one of them.  The groups taken, by 64 bits; 0 where the experts are more than
// a warp's lanes.
template <class T, int VPL>
__device__ __forceinline__ uint32_t scored_border_64(const ScoredParams &p, const T *row, uint32_t cand, uint32_t taken,
                                                     uint32_t border, double m, double sum)
{
    const int lane = threadIdx.x & 31;
    if (__reduce_add_sync(0xffffffffu, __popc(cand)) > 32) return 0;
    int n = 0, mine = -1;
#pragma unroll 1
    for (int j = 0; j < VPL; ++j)
        for (uint32_t lanes = __ballot_sync(0xffffffffu, cand >> j & 1u); lanes; lanes &= lanes - 1, ++n)
            if (lane == n) mine = (__ffs(lanes) - 1) * VPL + j;
    const uint64_t key = mine >= 0 ? scored_key(scored_c_64(p, scored_logit(row, mine), mine, m, sum)) : kKey64None;
    uint64_t a1 = kKey64None, a2 = kKey64None;  // of group `lane`
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const uint64_t k = __shfl_sync(0xffffffffu, key, i);
        if (__shfl_sync(0xffffffffu, mine, i) / p.per == lane) scored_two(a1, a2, k);
    }
    const bool open = border >> lane & 1u;
    const uint64_t score = !open ? kKey64None
                           : p.two && a2 > kKey64None ? scored_key(scored_value(a1) + scored_value(a2))
                                                      : a1;
    return (taken & ~border) | scored_groups(score, kKey64None, p.groups, __popc(taken & border));
}

// Choice and weights of a block's tokens; their masks; one cluster: everything.
// VPL: experts per lane (E <= 32 VPL), their logits in runs of V (16 bytes at most) where rows
// start on such.
template <class T, int VPL>
__global__ void __launch_bounds__(kScoredThreads, VPL <= 8 ? 2 : 1) moe_choose_scored_kernel(const ScoredParams sp)
{
    constexpr int V = VPL < 16 / int(sizeof(T)) ? VPL : 16 / int(sizeof(T));
    struct alignas(V * sizeof(T)) Run {
        T v[V];
    };
    constexpr float kNone = -__builtin_huge_valf();
    const RouteParams &p = sp.r;
    extern __shared__ uint2 mask[];  // [E], then first[E + 1], start[E], experts[kTB * k]
    overlap_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * VPL;
    const bool one_cluster = !p.counts && !p.packed_counts;
    int *first = reinterpret_cast<int *>(mask + p.E);
    int *start = first + p.E + 1;
    int *chosen = start + p.E;
    __shared__ int again[kTB], again_count;  // tokens to do again
    __shared__ float2 softmax[kTB];          // a token's largest logit and sum, where weights need them
    __shared__ float2 lists[kScoredThreads / 32][32];  // a warp's candidates: c, expert
    for (int e = threadIdx.x; e < p.E; e += kScoredThreads) mask[e] = make_uint2(0, 0);
    if (threadIdx.x == 0) again_count = 0;
    // (through shared memory: lanes VPL floats apart would take a line each)
    __shared__ float biases[32 * VPL + VPL];
    if (sp.bias)
        for (int e = threadIdx.x; e < p.E; e += kScoredThreads) biases[e + e / 32] = sp.bias[e];
    __syncthreads();
    float bias[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) bias[j] = sp.bias && e0 + j < p.E ? biases[e0 + j + (e0 + j) / 32] : 0.0f;
    bool any = false;
#pragma unroll
    for (int j = 0; j < VPL; ++j) any |= bias[j] != 0.0f;
    const bool biased = __any_sync(0xffffffffu, any);
    const int t0 = blockIdx.x * p.tb;
    const int mine = min(p.tb, p.T - t0);  // (t0 + tb may pass 2^31)
    const bool grouped = sp.groups > 1;
    // groups of whole lanes, a power of two of them
    const int lanes = sp.per / VPL;
    const bool runs = sp.per % VPL == 0 && (lanes & (lanes - 1)) == 0;
    // up to so many choices the candidates of one search mostly fit a warp's lanes (4096 x 512,
    // 32 choices: 39 us with the search first, 35.5 without)
    const bool few = p.k <= 16;
    const bool scores = biased || (grouped && sp.two);  // every expert's is needed
    constexpr int kWarps = kScoredThreads / 32;
    // The weights of the chosen of token i (the same in `per` lanes, a power of two).
    const auto weigh = [&](int i, int per) {
        const int q = lane & (per - 1);
        const int64_t t = t0 + i;
        const bool there = i < mine && q < p.k;
        const int my_e = there ? chosen[i * p.k + q] : -1;
        const float x = my_e >= 0 ? scored_logit(static_cast<const T *>(p.logits) + t * p.E, my_e) : kNone;
        // The weight before the scale.  Renormalised ones need no score that could underflow:
        // softmax from the largest chosen logit, sigmoids times e^-min(0, that).
        float w = 0.0f, total = i < mine ? softmax[i].y : 1.0f;
        if (p.normalize) {
            float most = x;
            for (int d = per / 2; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
            if (my_e >= 0) {
                if (!sp.sigmoid) w = expf(x - most);
                else if (x > 0.0f) w = scored_sigmoid(x);
                else w = __fdiv_rn(expf(x - fminf(most, 0.0f)), 1.0f + expf(x));
            }
            total = w;
            for (int d = per / 2; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
        } else if (my_e >= 0) {
            w = sp.sigmoid ? scored_sigmoid(x) : expf(x - softmax[i].x);
        }
        if (there) {
            p.experts[t * p.k + q] = my_e;
            p.weights[t * p.k + q] = my_e >= 0 ? sp.scale * __fdiv_rn(w, total) : 0.0f;
            if (my_e >= 0) atomicOr(i < 32 ? &mask[my_e].x : &mask[my_e].y, 1u << (i & 31));
        }
    };
    // a token's at once, or (more than two tokens a warp) after the last one (2048 x 256: 11.9 us
    // at once, 13.3 after; 16384 x 256: 32.1 and 29.2)
    const bool at_once = p.tb <= 2 * kWarps;
    for (int i = warp; i < mine; i += kWarps) {
        const int64_t t = t0 + i;
        const T *row = static_cast<const T *>(p.logits) + t * p.E;
        float c[VPL], s[VPL];
        float m = kNone;
#pragma unroll
        for (int j = 0; j < VPL; j += V) {
            Run run;
            if (sp.vec && e0 + j < p.E) {  // (E is a multiple of V)
                run = *reinterpret_cast<const Run *>(row + e0 + j);
            } else {
#pragma unroll
                for (int q = 0; q < V; ++q) run.v[q] = e0 + j + q < p.E ? row[e0 + j + q] : T(kNone);
            }
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float v = moe_float(run.v[q]);
                c[j + q] = v != v ? kNone : v + 0.0f;
                m = fmaxf(m, c[j + q]);
            }
        }
        // softmax: the largest logit and the sum over all experts; a row with +inf has no scores
        float sum = 1.0f;
        if (!sp.sigmoid) {
            m = route_value(__reduce_max_sync(0xffffffffu, route_key(m)));
            if (!(m < CUDART_INF_F)) {
#pragma unroll
                for (int j = 0; j < VPL; ++j) c[j] = kNone;
            }
            if (scores || !p.normalize) {
                sum = 0.0f;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    s[j] = !(c[j] > kNone) ? 0.0f : p.normalize ? __expf(c[j] - m) : expf(c[j] - m);
                    sum += s[j];
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            }
        }
        // Two c that are farther apart than slack + 2^-22 |c| are in order: twice the error of
        // one, of sigmoids 1.63 2^-22, of softmax 24.3 2^-23 of the largest score (an
        // exponential's 2 + 1.173 |x - m| ulp and |x - m| 2^-24 count e^(x - m), the sum takes
        // VPL + 5 roundings), and of the addition 2^-24 |c|.
        float slack = 0x1.ap-21f;
        if (scores) {
            const float inv = __fdiv_rn(1.0f, sum);
            if (!sp.sigmoid) slack = 0x1p-17f * inv;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                s[j] = !(c[j] > kNone) ? 0.0f : sp.sigmoid ? scored_sigmoid_fast(c[j]) : s[j] * inv;
                if (biased && c[j] > kNone) {
                    const float v = s[j] + bias[j];
                    c[j] = v > kNone ? v : kNone;  // (not NaN)
                }
            }
        }
        bool near = false;
        if (grouped) {
            float score = kNone, slip = 0.0f;  // of group `lane`
            if (runs) {
                float a1 = kNone, a2 = kNone;
                if (sp.two && !biased) {
#pragma unroll
                    for (int j = 0; j < VPL; ++j) scored_two(a1, a2, c[j] > kNone ? s[j] : kNone);
                } else {
#pragma unroll
                    for (int j = 0; j < VPL; ++j) scored_two(a1, a2, c[j]);
                }
                for (int d = 1; d < lanes; d <<= 1) {
                    const float b1 = __shfl_xor_sync(0xffffffffu, a1, d), b2 = __shfl_xor_sync(0xffffffffu, a2, d);
                    scored_join(a1, a2, b1, b2);
                }
                const float mine_score = scored_group(a1, a2, sp.two);
                score = __shfl_sync(0xffffffffu, mine_score, (lane * lanes) & 31);
                if (scores) slip = __shfl_sync(0xffffffffu, scored_slip(a1, a2, sp.two, slack, biased), (lane * lanes) & 31);
                if (lane >= sp.groups) score = kNone;
            } else {
                for (int g = 0; g < sp.groups; ++g) {
                    float a1 = kNone, a2 = kNone;
                    const int from = g * sp.per - e0, to = from + sp.per;
#pragma unroll
                    for (int j = 0; j < VPL; ++j)
                        if (j >= from && j < to && c[j] > kNone) scored_two(a1, a2, sp.two && !biased ? s[j] : c[j]);
#pragma unroll
                    for (int d = 16; d; d >>= 1) {
                        const float b1 = __shfl_xor_sync(0xffffffffu, a1, d), b2 = __shfl_xor_sync(0xffffffffu, a2, d);
                        scored_join(a1, a2, b1, b2);
                    }
                    if (lane == g) {
                        score = scored_group(a1, a2, sp.two);
                        slip = scored_slip(a1, a2, sp.two, slack, biased);
                    }
                }
            }
            uint32_t taken = scored_groups(score, kNone, sp.groups, sp.group_k);
            if (scores) {
                // the least that a group taken, and the most that one left, may be worth
                const bool in = taken >> lane & 1u, out = !in && lane < sp.groups && score > kNone;
                const float low = fmaxf(score - slip, kNone), high = score + slip;  // (+inf less +inf: -inf)
                const float least = route_value(__reduce_min_sync(0xffffffffu, in ? route_key(low) : 0xFF800000u));
                const float most = route_value(__reduce_max_sync(0xffffffffu, out ? route_key(high) : kKeyNone));
                if (most > kNone && !(least > most)) {
                    const uint32_t border = __ballot_sync(0xffffffffu, (in && !(low > most)) || (out && !(high < least)));
                    // their experts that may be the largest, or the two largest
                    uint32_t cand = 0;
                    for (uint32_t open = border; open; open &= open - 1) {
                        const int g = __ffs(open) - 1, from = g * sp.per - e0, to = from + sp.per;
                        if (!biased) {
#pragma unroll 1
                            for (int n = 0; n < 2; ++n) {
                                float a = kNone;
                                int at = 0;
#pragma unroll
                                for (int j = 0; j < VPL; ++j)
                                    if (j >= from && j < to && !(cand >> j & 1u) && c[j] > a) {
                                        a = c[j];
                                        at = j;
                                    }
                                const uint32_t local = route_key(a), top = __reduce_max_sync(0xffffffffu, local);
                                if (top <= kKeyNone) break;
                                if (lane == __ffs(__ballot_sync(0xffffffffu, local == top)) - 1) cand |= 1u << at;
                            }
                            continue;
                        }
                        float a1 = kNone, a2 = kNone;
#pragma unroll
                        for (int j = 0; j < VPL; ++j)
                            if (j >= from && j < to && c[j] > kNone) scored_two(a1, a2, c[j]);
#pragma unroll
                        for (int d = 16; d; d >>= 1) {
                            const float b1 = __shfl_xor_sync(0xffffffffu, a1, d), b2 = __shfl_xor_sync(0xffffffffu, a2, d);
                            scored_join(a1, a2, b1, b2);
                        }
                        const float least_of = sp.two ? a2 : a1;
#pragma unroll
                        for (int j = 0; j < VPL; ++j)
                            if (j >= from && j < to && c[j] > kNone &&
                                !(least_of - c[j] > slack + 0x1p-22f * fabsf(least_of)))
                                cand |= 1u << j;
                    }
                    const double sum64 = sp.sigmoid ? 1.0 : scored_sum_64<T, VPL>(sp, row, m);
                    taken = scored_border_64<T, VPL>(sp, row, cand, taken, border, m, sum64);
                    near = taken == 0;
                }
            }
            if (runs) {
                const bool in = lane < sp.groups * lanes && (taken >> lane / lanes & 1u);
#pragma unroll
                for (int j = 0; j < VPL; ++j) c[j] = in ? c[j] : kNone;
            } else {
                int g = e0 / sp.per, left = (g + 1) * sp.per - e0;  // experts until the next group
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    if (left == 0) {
                        ++g;
                        left = sp.per;
                    }
                    --left;
                    if (g >= 32 || !(taken >> g & 1u)) c[j] = kNone;
                }
            }
        }
        // lane n's expert and c by falling c: the k largest and, with a bias, those left that the
        // last of them does not surely exceed (some more do not matter)
        int my_e = -1, n = 0;
        float my_c = kNone;
        const auto apart = [&](float a, float b) { return a - b > slack + 0x1p-22f * fabsf(a); };
        // The k-th largest of the lanes' largest is at most the k-th largest of all: what is
        // not below it are the candidates, a few more than k.
        uint32_t cand = 0;
        int end = 0;
        n = 33;
        if (few) {
            float most = kNone;
#pragma unroll
            for (int j = 0; j < VPL; ++j) most = fmaxf(most, c[j]);
            uint32_t left = route_key(most), least = 0;
            for (int i = 0; i < p.k; ++i) {
                least = __reduce_max_sync(0xffffffffu, left);
                if (least <= kKeyNone) break;
                left = left == least ? 0 : left;
            }
            float cut = least > kKeyNone ? route_value(least) : kNone;
            if (biased) cut -= slack + 0x1p-22f * fabsf(cut);
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (c[j] > kNone && !(c[j] < cut)) cand |= 1u << j;
            end = __popc(cand);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, end, d);
                if (lane >= d) end += o;
            }
            n = __shfl_sync(0xffffffffu, end, 31);
        }
        if (n <= 32) {
            float2 *list = lists[warp];
            int at = end - __popc(cand);
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (cand >> j & 1u) list[at++] = make_float2(c[j], __int_as_float(e0 + j));
            __syncwarp();
            const float2 own = lane < n ? list[lane] : make_float2(kNone, 0.0f);
            int rank = 0;  // (in the order of the experts: of equal ones the first)
            for (int i = 0; i < n; ++i) {
                const float other = __shfl_sync(0xffffffffu, own.x, i);
                rank += other > own.x || (other == own.x && i < lane) ? 1 : 0;
            }
            __syncwarp();
            if (lane < n) list[rank] = own;
            __syncwarp();
            if (lane < n) {
                my_c = list[lane].x;
                my_e = __float_as_int(list[lane].y);
            }
            __syncwarp();  // read before the next token's
        } else {
            // one at a time
            n = 0;
            // A lane's two largest that are not taken, looked for again once both are: few lanes
            // hold more than two of a token's choices.
            float a1 = kNone, a2 = kNone;
            int at1 = 0, at2 = 0, held = 2;
            uint32_t used = 0;
            const auto look = [&] {
                a1 = a2 = kNone;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    const float v = used >> j & 1u ? kNone : c[j];
                    const bool first_of = v > a1, second = v > a2;
                    a2 = first_of ? a1 : second ? v : a2;
                    at2 = first_of ? at1 : second ? j : at2;
                    a1 = first_of ? v : a1;
                    at1 = first_of ? j : at1;
                }
            };
            look();
            // lane n keeps choice n; those left that the last one does not surely exceed join the list
            float last = kNone;
            uint32_t local = route_key(a1), top = __reduce_max_sync(0xffffffffu, local);
            for (; top > kKeyNone; ++n) {
                if (n >= p.k) {
                    if (!biased) break;
                    if (n == p.k) last = __shfl_sync(0xffffffffu, my_c, p.k - 1);
                    if (apart(last, route_value(top))) break;
                    near |= n == 32;  // (more than the list holds)
                    if (n == 32) break;
                }
                const int owner = __ffs(__ballot_sync(0xffffffffu, local == top)) - 1;
                const int e = owner * VPL + __shfl_sync(0xffffffffu, at1, owner);
                if (lane == n) {
                    my_e = e;
                    my_c = route_value(top);
                }
                if (lane == owner) {
                    used |= 1u << at1;
                    if (--held) {
                        a1 = a2;
                        at1 = at2;
                    } else {
                        look();
                        held = 2;
                    }
                    local = route_key(a1);
                }
                top = __reduce_max_sync(0xffffffffu, local);
            }
        }
        if (biased) {
            // Neighbours nearer than the rounding, but for those that are equal in both parts: among
            // the chosen, and behind them as far as the last one chosen does not surely exceed (of
            // equal ones there another may be the larger).
            const float x = my_e >= 0 ? scored_logit(row, my_e) : kNone;
            const float b = my_e >= 0 ? sp.bias[my_e] : 0.0f, v = my_c;
            const float x2 = __shfl_down_sync(0xffffffffu, x, 1), b2 = __shfl_down_sync(0xffffffffu, b, 1);
            const float v2 = __shfl_down_sync(0xffffffffu, v, 1), last = __shfl_sync(0xffffffffu, v, p.k - 1);
            const bool unsure = lane + 1 < n && (lane + 1 < p.k || !apart(last, v2)) && !apart(v, v2) &&
                                !(x == x2 && b == b2);
            if (__any_sync(0xffffffffu, unsure)) {
                const double sum64 = sp.sigmoid ? 1.0 : scored_sum_64<T, VPL>(sp, row, m);
                my_e = scored_order_64(sp, my_e, x, n, m, sum64);
            }
        }
        if (near) {
            if (lane == 0) again[atomicAdd(&again_count, 1)] = i;
            continue;
        }
        if (lane < p.k) chosen[i * p.k + lane] = my_e;
        if (lane == 0) softmax[i] = make_float2(m, sum);
        if (at_once) {
            __syncwarp();
            weigh(i, 32);
        }
    }
    __syncthreads();
    for (int n = warp; n < again_count; n += kWarps) {
        const int i = again[n];
        const T *row = static_cast<const T *>(p.logits) + static_cast<int64_t>(t0 + i) * p.E;
        float m = kNone, sum = 1.0f;
        if (!sp.sigmoid && !p.normalize) {
            for (int e = lane; e < p.E; e += 32) m = fmaxf(m, scored_logit(row, e));
            m = route_value(__reduce_max_sync(0xffffffffu, route_key(m)));
            sum = 0.0f;
            for (int e = lane; e < p.E; e += 32) sum += expf(scored_logit(row, e) - m);
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        }
        const int my_e = scored_choose_64<T, VPL>(sp, row, biased);
        if (lane < p.k) chosen[i * p.k + lane] = my_e;
        if (lane == 0) softmax[i] = make_float2(m, sum);
    }
    __syncthreads();
    if (!at_once || again_count) {
        // several tokens a warp
        int per = 1;
        while (per < p.k) per *= 2;
        const int tokens = 32 / per;
        for (int i0 = warp * tokens; i0 < mine; i0 += kWarps * tokens) weigh(i0 + lane / per, per);
    }
    overlap_release();
    __syncthreads();
    if (!one_cluster) {
        route_counts(p, mask);
        return;
    }
    route_finish<kScoredThreads>(p, mask, first, start, chosen);
}

template <class T, int VPL>
static int launch_scored_vpl(ScoredParams p, int smem, cudaStream_t stream)
{
    constexpr int V = VPL < 16 / int(sizeof(T)) ? VPL : 16 / int(sizeof(T));
    p.vec = p.r.E % V == 0 && reinterpret_cast<uintptr_t>(p.r.logits) % (V * sizeof(T)) == 0;
    const auto kernel = moe_choose_scored_kernel<T, VPL>;
    if (p.r.counts || p.r.packed_counts)
        return launch_overlapped(kernel, dim3(p.r.blocks), dim3(kScoredThreads), smem + kTB * p.r.k * 4, stream, p);
    int cluster = 1;
    while (cluster < p.r.blocks) cluster *= 2;  // (blocks without tokens fill it up)
    return launch_overlapped_clusters(kernel, dim3(cluster), cluster, dim3(kScoredThreads), smem, stream, p);
}

template <class T>
static int launch_scored(const ScoredParams &p, int smem, cudaStream_t stream)
{
    if (p.r.E <= 64) return launch_scored_vpl<T, 2>(p, smem, stream);
    if (p.r.E <= 128) return launch_scored_vpl<T, 4>(p, smem, stream);
    if (p.r.E <= 256) return launch_scored_vpl<T, 8>(p, smem, stream);
    if (p.r.E <= 512) return launch_scored_vpl<T, 16>(p, smem, stream);
    return launch_scored_vpl<T, 32>(p, smem, stream);
}

int launch_moe_route_scored(const MoeScoredCall &c, cudaStream_t stream)
{
    RouteParams p{};
    p.logits = c.route.logits;
    p.experts = c.route.experts;
    p.weights = c.route.weights;
    p.offsets = c.route.offsets;
    p.tokens = c.route.tokens;
    p.slots = c.route.slots;
    p.T = c.route.T;
    p.E = c.route.E;
    p.k = c.route.k;
    p.normalize = c.route.normalize ? 1 : 0;
    // blocks in whole waves of two on every SM
    const int64_t wave = 2 * sm_count(), waves = (int64_t(p.T) + wave * kTB - 1) / (wave * kTB);
    const int tb = std::max(16, static_cast<int>((p.T + waves * wave - 1) / std::max<int64_t>(1, waves * wave)));
    const auto choose = [&](const RouteParams &q, int smem) {
        const ScoredParams sp{q, c.bias, c.score == 1, c.groups, q.E / c.groups, c.group_k, c.group_top == 2, c.scale, 0};
        return c.route.x_type == 0   ? launch_scored<float>(sp, smem, stream)
               : c.route.x_type == 1 ? launch_scored<__nv_bfloat16>(sp, smem, stream)
                                     : launch_scored<__half>(sp, smem, stream);
    };
    // One cluster is eight blocks: for more than 2^16 scores (or 512 tokens) many blocks are
    // faster in spite of a second launch (us a call, one cluster and two launches, softmax alone:
    // 256 x 256 9.0 and 10.6, 512 x 128 10.6 and 10.5, 512 x 256 12.2 and 10.6, 512 x 1024 24.6 and
    // 12.6; sigmoids, a bias, 8 groups by two: 256 x 128 10.3 and 11.2, 256 x 256 12.3 and 10.9, 512
    // x 128 15.2 and 11.3, 512 x 256 18.4 and 10.8, 512 x 1024 39.7 and 17.0.  In a captured graph,
    // without the host's time, two launches gain from half of that size on: 512 x 128 10.2 and 6.8,
    // 14.8 and 8.1).
    return route_launch(p, stream, choose, tb, std::min(kClusterBlocks * kTB, (1 << 16) / std::max(1, p.E)));
}

// ---------------------------------------------------------------- gradient
__device__ __forceinline__ void scored_out(float *o, float v) { *o = v; }
__device__ __forceinline__ void scored_out(__nv_bfloat16 *o, float v) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void scored_out(__half *o, float v) { *o = __float2half_rn(v); }

// With u the weights before the scale and g their gradient:
//   renormalised  dx_i = scale u_i (g_i - sum_j g_j u_j), times sigmoid(-x_i) for sigmoids
//   sigmoids      dx_i = scale u_i sigmoid(-x_i) g_i
//   softmax       dx_e = scale (sum of the g of e's pairs, times u_e, - p_e sum_j g_j u_j)
// A warp per token: lane j the pair j, then the row (zeros, or the last line's second part)
// in runs of V, then the chosen logits' own values over it.  The row is written, and read
// where every logit has a gradient: 16384 x 256 float32 sigmoids, renormalised, 7 us (17 MB
// written; the host's time of a call), 10 from a cold cache.
template <class T, int V>
__global__ void __launch_bounds__(256) moe_scored_grad_kernel(const T *logits, const int *experts, const float *dweights,
                                                              T *dlogits, int Tn, int E, int k, int sigmoid, int normalize,
                                                              float scale)
{
    struct alignas(V * sizeof(T)) Run {
        T v[V];
    };
    constexpr float kNone = -__builtin_huge_valf();
    overlap_wait();
    const int lane = threadIdx.x & 31;
    const bool dense = !sigmoid && !normalize;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < Tn; t += step) {
        const T *row = logits + t * E;
        T *out = dlogits + t * E;
        int e = lane < k ? experts[t * k + lane] : -1;
        float g = lane < k ? dweights[t * k + lane] : 0.0f;
        float x = e >= 0 && e < E ? scored_logit(row, e) : kNone;
        if (!(x > kNone)) {  // no choice, or one that has no weight
            e = -1;
            g = 0.0f;
        }
        // a softmax row with +inf has no scores (renormalised, the other logits are not read: only
        // where it is named)
        if (!sigmoid && __any_sync(0xffffffffu, x == CUDART_INF_F)) {
            e = -1;
            g = 0.0f;
        }
        float m = 0.0f, inv = 0.0f;
        if (dense) {
            // the row's largest and the sum, a lane's running ones joined
            m = kNone;
            float sum = 0.0f;
            for (int i = lane * V; i < E; i += 32 * V) {
                const Run run = *reinterpret_cast<const Run *>(row + i);
                float v[V], most = m;
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    v[q] = moe_float(run.v[q]);
                    if (v[q] != v[q]) v[q] = kNone;
                    most = fmaxf(most, v[q]);
                }
                if (most > kNone) {
                    sum = m > kNone ? sum * expf(m - most) : 0.0f;
#pragma unroll
                    for (int q = 0; q < V; ++q) sum += expf(v[q] - most);
                    m = most;
                }
            }
            const float most = route_value(__reduce_max_sync(0xffffffffu, route_key(m)));
            sum = m > kNone ? sum * expf(m - most) : 0.0f;
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            m = most;
            if (m > kNone && m < CUDART_INF_F) {
                inv = __fdiv_rn(1.0f, sum);
            } else {  // no scores: nothing was chosen
                e = -1;
                g = 0.0f;
            }
        }
        // u of the pair, and how much of its score's gradient reaches the logit
        float u = 0.0f, part = 1.0f;
        if (sigmoid) part = e >= 0 ? scored_sigmoid(-x) : 0.0f;
        if (normalize) {
            const float most = route_value(__reduce_max_sync(0xffffffffu, route_key(e >= 0 ? x : kNone)));
            if (e >= 0) {
                if (!sigmoid) u = expf(x - most);
                else if (x > 0.0f) u = scored_sigmoid(x);
                else u = __fdiv_rn(expf(x - fminf(most, 0.0f)), 1.0f + expf(x));
            }
            float total = u;
#pragma unroll
            for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
            if (e >= 0) u = __fdiv_rn(u, total);
        } else if (e >= 0) {
            u = sigmoid ? scored_sigmoid(x) : expf(x - m) * inv;
        }
        float mean = 0.0f;
        if (!sigmoid || normalize) {
            mean = g * u;
#pragma unroll
            for (int d = 16; d; d >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, d);
        }
        float d = scale * u * part * (g - (normalize ? mean : 0.0f));
        // an expert twice in a token: the first of its pairs writes the sum
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && (same & (same - 1))) {
            float all = 0.0f;
            for (int j = 0; j < k; ++j) {
                const float o = __shfl_sync(same, d, j);
                if (same >> j & 1u) all += o;
            }
            d = all;
        }
        if (dense) d -= scale * u * mean;
        const float of_row = scale * mean;
        for (int i = lane * V; i < E; i += 32 * V) {
            Run run;
            if (dense && inv > 0.0f) {
                const Run in = *reinterpret_cast<const Run *>(row + i);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float v = moe_float(in.v[q]);
                    scored_out(&run.v[q], v > kNone ? -(expf(v - m) * inv) * of_row : 0.0f);
                }
            } else {
#pragma unroll
                for (int q = 0; q < V; ++q) scored_out(&run.v[q], 0.0f);
            }
            *reinterpret_cast<Run *>(out + i) = run;
        }
        __syncwarp();  // the row before the values of the chosen ones
        if (e >= 0 && lane == __ffs(same) - 1) scored_out(out + e, d);
    }
    overlap_release();
}

template <class T, int V>
static int launch_grad(const MoeScoredGradCall &c, cudaStream_t stream)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(c.logits) | reinterpret_cast<uintptr_t>(c.dlogits);
    if constexpr (V > 1)
        if (at % (V * sizeof(T)) != 0 || c.E % V != 0) return launch_grad<T, V / 2>(c, stream);
    const int64_t blocks = std::min<int64_t>((int64_t(c.T) + 7) / 8, int64_t(sm_count()) * 8);
    return launch_overlapped(moe_scored_grad_kernel<T, V>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                             static_cast<const T *>(c.logits), c.experts, c.dweights, static_cast<T *>(c.dlogits), c.T, c.E,
                             c.k, c.score == 1 ? 1 : 0, c.normalize ? 1 : 0, c.scale);
}

int launch_moe_route_scored_grad(const MoeScoredGradCall &c, cudaStream_t stream)
{
    switch (c.x_type) {
    case 0: return launch_grad<float, 4>(c, stream);
    case 1: return launch_grad<__nv_bfloat16, 8>(c, stream);
    default: return launch_grad<__half, 8>(c, stream);
    }
}

}  // namespace igemm
