// Microscaled 4-bit floating-point GEMM, dense or grouped by expert:
//
//   C[m,n] = alpha * sum_k (a[m,k] sfa[m,k/B]) (b[n,k] sfb[n,k/B])
//
// with e2m1 codes packed two per byte and one scale per row and B = 32 k (ue8m0,
// "mx") or 16 k (ue4m3, "nv"), float32 accumulation in tensor memory.  The
// weights B are the MMA's M side (128 rows per CTA) and the activations its N
// side: one kernel then serves a single token (N = 16) and a prompt (N = 256 on a
// CTA pair), the N of a ragged last tile is set per tile in the instruction
// descriptor, and a lane of the accumulator is an output column, so C rows are
// written 32 consecutive columns at a time whatever their alignment.
//
// The scale of a row's 16 bytes (512 k mx, 256 k nv: one "unit") lands with its own
// small TMA box, row-major as the caller has it, at any row (a group starts
// anywhere).  The tensor core wants the words of 128 rows across 4 columns of
// all four TMEM lane quadrants, so four warps, one per quadrant, read the rows'
// 16 bytes (conflict-free) and store the 4 words of every row with two TMEM
// stores per unit; no layout pass runs over the scales.
//
// Warps 0-3 epilogue, 4-7 scales, 8 TMA producer, 9 MMA issue.  Persistent
// CTAs (or CTA pairs, or clusters that split k).  Every wait is bounded.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "ptx.cuh"

namespace igemm {

constexpr int kFp4MaxExperts = 1024;

enum Fp4OutType : int { kOutF32 = 0, kOutBf16 = 1, kOutF16 = 2 };

struct Fp4Params {
    void *C;               // [rows, N] row-major
    int c_type;            // Fp4OutType
    const float *alpha;    // [experts] or null (1)
    const int *offsets;    // [experts + 1] rows of each group, or null: one group of all rows
    int rows, N, experts;
    int k_steps;           // MMA steps of 64 k: ceil(K / 64)
    int k_blocks;          // scale bytes in use per row
    int stages;            // pipeline stages of 512 k: ceil(K / 512)
    int units;             // scale units: ceil(K / 512) (mx), ceil(K / 256) (nv)
    int qt;                // activation rows per tile (<= BN)
    int p_tiles;           // tiles of 128 weight rows (pair: of 256)
    int group_p;           // tiles run in groups of group_p weight tiles (fastest) by every activation tile
    int cs;                // CTAs of a cluster that split k (1: none)
    int stages_per_slice;
    int code_stages, scale_stages;
    int off_scales, off_red, off_bars;  // shared-memory offsets after the code stages
    int *status;
    unsigned long long limit_ns;
};

template <bool NV_, int BN_, bool PAIR_>
struct Fp4Cfg {
    static constexpr bool NV = NV_;
    static constexpr bool PAIR = PAIR_;
    static constexpr int BN = BN_;                     // most activation rows per tile
    static constexpr int CL = PAIR ? 2 : 1;
    static constexpr int kQBox = BN / CL;              // activation rows this CTA loads
    static constexpr int kU = NV ? 2 : 1;              // scale units per stage
    static constexpr int kBoxP = 128 * 128;            // bytes of 256 k
    static constexpr int kBoxQ = kQBox * 128;
    // a stage holds 512 k, two boxes of each operand: its 8 MMAs keep the tensor
    // pipe busy while the issuing warp goes through its waits and commits
    static constexpr int kStage = 2 * (kBoxP + kBoxQ);
    static constexpr int kScaleStage = (128 + BN) * 16;
    static constexpr int kQCols = BN <= 128 ? 4 : BN / 32;   // TMEM columns of one word of every activation row
    static constexpr int kSfCols = 16 + 4 * kQCols;    // TMEM columns of one unit's scales
    static constexpr int kSfSlots = BN == 256 && !NV ? 2 : 4;
    // two accumulators of BN columns; with BN = 256 the second starts before
    // the first ends (kOverlap columns), so that the scales fit beside them
    static constexpr int kAcc1 = BN == 256 ? 512 - kSfSlots * kSfCols - BN : BN;
    static constexpr int kOverlap = BN - kAcc1;
    static constexpr int kSf0 = kAcc1 + BN;
    static constexpr int kTmemUse = kSf0 + kSfSlots * kSfCols;
    static constexpr int kTmemCols = kTmemUse <= 128 ? 128 : kTmemUse <= 256 ? 256 : 512;
    static constexpr int kRedBufs = BN <= 32 ? 2 : 1;
    static constexpr int kRedBytes = kRedBufs * BN * 512;  // split k: partial tiles of the cluster's CTAs
    static constexpr int kMaxStages = 16;
    static constexpr int kNumBars = 4 * kMaxStages + 2 * kSfSlots + 4 + 1 + 4;
    static constexpr int kTailBytes = 8 * kNumBars + 64 + 4 * (kFp4MaxExperts + 1);
    static constexpr int kNAlign = PAIR ? 32 : 16;
    static constexpr int kThreads = 320;
    static_assert(kQBox % 8 == 0 && kStage % 1024 == 0, "1024-byte aligned operand tiles");
    static_assert(kTmemUse <= 512 && kOverlap >= 0 && kOverlap % 96 == 0, "TMEM budget");
    static_assert(!PAIR || BN == 256, "the pair form is built for 256 activation rows");
};

struct Fp4Tile {
    int e;        // expert
    int p0;       // first weight row within the expert of this CTA
    int q0;       // first activation row (of all rows)
    int nq;       // activation rows of the tile
};

// Tile t: expert by binary search in the running tile counts, then the grouped
// order of its weight and activation tiles.
template <class Cfg>
__device__ __forceinline__ Fp4Tile fp4_tile(const Fp4Params &prm, const int *first_tile, int t, int rank)
{
    Fp4Tile x;
    int begin = 0, count = prm.rows, r = t;
    x.e = 0;
    if (prm.offsets) {
        int lo = 0, hi = prm.experts;  // first_tile[lo] <= t < first_tile[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_tile[mid] <= t) lo = mid;
            else hi = mid;
        }
        x.e = lo;
        r = t - first_tile[lo];
        begin = min(max(__ldg(prm.offsets + lo), 0), prm.rows);
        count = min(max(__ldg(prm.offsets + lo + 1), begin), prm.rows) - begin;
    }
    const int q_tiles = (count + prm.qt - 1) / prm.qt;
    const int per_group = prm.group_p * q_tiles;
    const int grp = r / per_group;
    const int first = grp * prm.group_p;
    const int gsize = min(prm.p_tiles - first, prm.group_p);
    r -= grp * per_group;
    const int qi = r / gsize;
    x.p0 = ((first + r - qi * gsize) * Cfg::CL + rank) * 128;
    x.q0 = begin + qi * prm.qt;
    x.nq = min(count - qi * prm.qt, prm.qt);
    return x;
}

__device__ __forceinline__ bool fp4_warp_wait(uint64_t *bar, uint32_t parity, const Watchdog &wd)
{
    const bool ok = wait_bounded(bar, parity, wd);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool fp4_warp_wait_cluster(uint64_t *bar, uint32_t parity, const Watchdog &wd)
{
    const bool ok = wait_bounded_cluster(bar, parity, wd);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void fp4_wait_drain(uint64_t *bar, uint32_t parity, unsigned long long limit_ns)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < limit_ns) {
    }
}

// Ring position: slot and phase parity, without divisions.
struct Fp4Ring {
    int slot = 0, n;
    uint32_t phase = 0;
    __device__ explicit Fp4Ring(int n_) : n(n_) {}
    __device__ void next()
    {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// The bytes of word `w` (scales 4 w ..) that lie below `n` scale bytes.
__device__ __forceinline__ uint32_t fp4_keep(uint32_t v, int left)
{
    return left >= 4 ? v : left <= 0 ? 0u : v & (0xFFFFFFFFu >> (8 * (4 - left)));
}

// `count` accumulator columns (rows m0 .. of C) of this lane's output column n.
template <int COUNT>
__device__ __forceinline__ void fp4_store(const Fp4Params &prm, const uint32_t (&v)[COUNT], float alpha, int64_t m0,
                                          int count, int n)
{
    if (n >= prm.N) return;
    const int64_t at = m0 * prm.N + n;
    if (prm.c_type == kOutF32) {
        float *c = static_cast<float *>(prm.C) + at;
#pragma unroll
        for (int j = 0; j < COUNT; ++j)
            if (j < count) c[static_cast<int64_t>(j) * prm.N] = __uint_as_float(v[j]) * alpha;
    } else if (prm.c_type == kOutBf16) {
        __nv_bfloat16 *c = static_cast<__nv_bfloat16 *>(prm.C) + at;
#pragma unroll
        for (int j = 0; j < COUNT; ++j)
            if (j < count) c[static_cast<int64_t>(j) * prm.N] = __float2bfloat16_rn(__uint_as_float(v[j]) * alpha);
    } else {
        __half *c = static_cast<__half *>(prm.C) + at;
#pragma unroll
        for (int j = 0; j < COUNT; ++j)
            if (j < count) c[static_cast<int64_t>(j) * prm.N] = __float2half_rn(__uint_as_float(v[j]) * alpha);
    }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    igemm_fp4_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                     const __grid_constant__ CUtensorMap mapSP, const __grid_constant__ CUtensorMap mapSQ,
                     const Fp4Params prm)
{
    constexpr bool NV = Cfg::NV, PAIR = Cfg::PAIR;
    constexpr int BN = Cfg::BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *codes = smem;
    uint8_t *scales = smem + prm.off_scales;
    float *red = reinterpret_cast<float *>(smem + prm.off_red);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + prm.off_bars);
    uint64_t *full = bars;                          // [stages] codes landed (pair: both CTAs', in the even CTA)
    uint64_t *empty = full + Cfg::kMaxStages;       // [stages] codes consumed (MMA commit)
    uint64_t *s_full = empty + Cfg::kMaxStages;     // [scale stages] scale bytes landed
    uint64_t *s_empty = s_full + Cfg::kMaxStages;   // [scale stages] ... read (4 scale warps)
    uint64_t *sf_ready = s_empty + Cfg::kMaxStages; // [slots] scales in TMEM (scale warps; pair: of both CTAs)
    uint64_t *sf_free = sf_ready + Cfg::kSfSlots;   // [slots] ... consumed (MMA commit)
    uint64_t *acc_full = sf_free + Cfg::kSfSlots;   // [2] accumulator complete (commit)
    uint64_t *acc_empty = acc_full + 2;             // [2] accumulator (its overlap) read by the epilogue warps
    uint64_t *mma_drain = acc_empty + 2;
    uint64_t *red_full = mma_drain + 1;             // [2] split k: every CTA's partials of this CTA's columns written
    uint64_t *red_empty = red_full + 2;             // [2] ... and every CTA's reads of what this CTA wrote done
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Cfg::kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *total_slot = reinterpret_cast<int *>(tmem_slot + 2);
    int *first_tile = reinterpret_cast<int *>(tmem_slot + 16);  // [experts + 1]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int cs = PAIR ? 1 : prm.cs;
    const int csize = PAIR ? 2 : cs;
    const int rank = csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int pr = PAIR ? rank : 0;                 // half of the pair's tile
    const int cid = blockIdx.x / csize, ncl = gridDim.x / csize;
    const bool leader = !PAIR || rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < prm.code_stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < prm.scale_stages; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_empty[s], 4);
        }
        for (int s = 0; s < Cfg::kSfSlots; ++s) {
            mbar_init(&sf_ready[s], 4 * Cfg::CL);
            mbar_init(&sf_free[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 4 * Cfg::CL);
            mbar_init(&red_full[b], 4 * cs);
            mbar_init(&red_empty[b], 4 * cs);
        }
        mbar_init(mma_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&mapP);
        tma_prefetch_map(&mapQ);
        tma_prefetch_map(&mapSP);
        tma_prefetch_map(&mapSQ);
    }
    if (warp == 9) {
        if constexpr (PAIR) {
            tmem_alloc_pair(tmem_slot, Cfg::kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, Cfg::kTmemCols);
            tmem_relinquish();
        }
    }
    if (warp == 0) {
        // running tile counts of the groups
        if (prm.offsets) {
            int run = 0;
            for (int e0 = 0; e0 < prm.experts; e0 += 32) {
                const int e = e0 + lane;
                int tiles = 0;
                if (e < prm.experts) {
                    const int b = min(max(__ldg(prm.offsets + e), 0), prm.rows);
                    const int n = min(max(__ldg(prm.offsets + e + 1), b), prm.rows) - b;
                    tiles = (n + prm.qt - 1) / prm.qt * prm.p_tiles;
                }
                int incl = tiles;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d) incl += o;
                }
                if (e < prm.experts) first_tile[e] = run + incl - tiles;
                run += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) {
                first_tile[prm.experts] = run;
                *total_slot = run;
            }
        } else if (lane == 0) {
            *total_slot = (prm.rows + prm.qt - 1) / prm.qt * prm.p_tiles;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (csize > 1) cluster_sync_all();  // the other CTAs' barriers are initialised
    const uint32_t tmem = *tmem_slot;
    const int tiles = *total_slot;
    const Watchdog wd{abort_flag, prm.status, prm.limit_ns};
    // this CTA's slice of k (split k: the cluster rank's), in stages
    const int k0 = PAIR ? 0 : min(rank * prm.stages_per_slice, prm.stages);
    const int k1 = PAIR ? prm.stages : min(k0 + prm.stages_per_slice, prm.stages);

    if (warp == 8) {
        // ------------------------------------------------------------ producer
        Fp4Ring cr(prm.code_stages), sr(prm.scale_stages);
        uint32_t issued = 0, last = 0, s_issued = 0, s_last = 0;
        bool ok = true;
        for (int t = cid; ok && t < tiles; t += ncl) {
            const Fp4Tile x = fp4_tile<Cfg>(prm, first_tile, t, pr);
            const int py = x.e * prm.N + x.p0;
            const int half = PAIR ? ((x.nq + Cfg::kNAlign - 1) & ~(Cfg::kNAlign - 1)) / 2 : 0;
            const int qy = x.q0 + pr * half;
            for (int k = k0; ok && k < k1; ++k) {
#pragma unroll
                for (int h = 0; h < Cfg::kU; ++h) {
                    const int u = k * Cfg::kU + h;
                    if (u >= prm.units) break;
                    if (!fp4_warp_wait(&s_empty[sr.slot], sr.phase ^ 1u, wd)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t *sc = scales + sr.slot * Cfg::kScaleStage;
                        mbar_arrive_expect_tx(&s_full[sr.slot], Cfg::kScaleStage);
                        tma_load_2d(sc, &mapSP, &s_full[sr.slot], u * 16, py);
                        tma_load_2d(sc + 128 * 16, &mapSQ, &s_full[sr.slot], u * 16, x.q0);
                    }
                    __syncwarp();
                    s_issued |= 1u << sr.slot;
                    s_last = (s_last & ~(1u << sr.slot)) | (sr.phase << sr.slot);
                    sr.next();
                }
                if (!ok || !fp4_warp_wait(&empty[cr.slot], cr.phase ^ 1u, wd)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    uint8_t *st = codes + cr.slot * Cfg::kStage;
                    if constexpr (PAIR) {
                        // both CTAs' bytes count on the even CTA's barrier
                        if (leader) mbar_arrive_expect_tx(&full[cr.slot], 2 * Cfg::kStage);
                        const uint32_t bar = cluster_map(smem_u32(&full[cr.slot]), 0u);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            tma_load_2d_pair(st + h * Cfg::kBoxP, &mapP, bar, (2 * k + h) * 128, py);
                            tma_load_2d_pair(st + 2 * Cfg::kBoxP + h * Cfg::kBoxQ, &mapQ, bar, (2 * k + h) * 128, qy);
                        }
                    } else {
                        mbar_arrive_expect_tx(&full[cr.slot], Cfg::kStage);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            tma_load_2d(st + h * Cfg::kBoxP, &mapP, &full[cr.slot], (2 * k + h) * 128, py);
                            tma_load_2d(st + 2 * Cfg::kBoxP + h * Cfg::kBoxQ, &mapQ, &full[cr.slot],
                                        (2 * k + h) * 128, qy);
                        }
                    }
                }
                __syncwarp();
                issued |= 1u << cr.slot;
                last = (last & ~(1u << cr.slot)) | (cr.phase << cr.slot);
                cr.next();
            }
        }
        // never leave with copies in flight, nor with an MMA commit on its way here
#pragma unroll 1
        for (int s = 0; s < prm.code_stages; ++s)
            if ((issued >> s) & 1u) {
                if (leader) fp4_wait_drain(&full[s], (last >> s) & 1u, prm.limit_ns);
                fp4_wait_drain(&empty[s], (last >> s) & 1u, prm.limit_ns);
            }
#pragma unroll 1
        for (int s = 0; s < prm.scale_stages; ++s)
            if ((s_issued >> s) & 1u) fp4_wait_drain(&s_full[s], (s_last >> s) & 1u, prm.limit_ns);
    } else if (warp == 9) {
        // ------------------------------------------------------------ MMA issuer
        if (leader) {
            Fp4Ring cr(prm.code_stages), fr(Cfg::kSfSlots);
            const uint64_t desc0 = sdesc_kmajor_sw128(smem_u32(codes));
            uint32_t nacc = 0;
            bool ok = true;
            for (int t = cid; ok && t < tiles; t += ncl, ++nacc) {
                const Fp4Tile x = fp4_tile<Cfg>(prm, first_tile, t, pr);
                const uint32_t nq = static_cast<uint32_t>((x.nq + Cfg::kNAlign - 1) & ~(Cfg::kNAlign - 1));
                const uint32_t idesc = idesc_fp4(128 * Cfg::CL, nq, NV);
                const uint32_t ab = nacc & 1u;
                const uint32_t d_tmem = tmem + ab * Cfg::kAcc1;
                if constexpr (Cfg::kOverlap > 0) {
                    // the tile before has left the columns that both accumulators use
                    if (nacc > 0 && !fp4_warp_wait(&acc_empty[ab ^ 1u], ((nacc - 1u) >> 1) & 1u, wd)) break;
                } else {
                    if (!fp4_warp_wait(&acc_empty[ab], ((nacc >> 1) & 1u) ^ 1u, wd)) break;
                }
                for (int k = k0; k < k1; ++k) {
                    if (!fp4_warp_wait(&full[cr.slot], cr.phase, wd)) {
                        ok = false;
                        break;
                    }
                    const uint64_t a0 = desc0 + static_cast<uint64_t>((cr.slot * Cfg::kStage) >> 4);
                    const uint64_t b0 = a0 + static_cast<uint64_t>((2 * Cfg::kBoxP) >> 4);
                    const int steps = prm.k_steps - 8 * k;
#pragma unroll
                    for (int h = 0; h < Cfg::kU; ++h) {
                        if (k * Cfg::kU + h >= prm.units) break;
                        if (!fp4_warp_wait(&sf_ready[fr.slot], fr.phase, wd)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sfp = tmem + Cfg::kSf0 + fr.slot * Cfg::kSfCols;
                        const uint32_t sfq = sfp + 16;
                        if (elect_one()) {
#pragma unroll
                            for (int q = 0; q < 8 / Cfg::kU; ++q) {  // MMA q of the unit
                                const int step = h * (8 / Cfg::kU) + q;
                                if (step < steps) {
                                    const int word = NV ? q : q / 2;  // a word holds 64 (nv) or 128 (mx) k
                                    const uint32_t id = NV ? 0u : 2u * (q & 1);
                                    const int box = step / 4, in = step % 4;
                                    mma_fp4<NV, PAIR>(d_tmem, a0 + static_cast<uint64_t>((box * Cfg::kBoxP >> 4) + 2 * in),
                                                      b0 + static_cast<uint64_t>((box * Cfg::kBoxQ >> 4) + 2 * in),
                                                      idesc | (id << 4) | (id << 29), sfp + 4 * word,
                                                      sfq + Cfg::kQCols * word, k > k0 || step > 0 ? 1u : 0u);
                                }
                            }
                            if constexpr (PAIR)
                                mma_commit_pair_multicast(&sf_free[fr.slot], 0x3);
                            else
                                mma_commit(&sf_free[fr.slot]);
                        }
                        __syncwarp();
                        fr.next();
                    }
                    if (!ok) break;
                    if (elect_one()) {
                        if constexpr (PAIR)
                            mma_commit_pair_multicast(&empty[cr.slot], 0x3);
                        else
                            mma_commit(&empty[cr.slot]);
                    }
                    __syncwarp();
                    cr.next();
                }
                if (ok && elect_one()) {
                    if constexpr (PAIR)
                        mma_commit_pair_multicast(&acc_full[ab], 0x3);
                    else
                        mma_commit(&acc_full[ab]);
                }
                __syncwarp();
            }
            if (elect_one()) {
                if constexpr (PAIR)
                    mma_commit_pair(mma_drain);
                else
                    mma_commit(mma_drain);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ scales into TMEM
        const uint32_t quad = static_cast<uint32_t>(warp & 3);
        const uint32_t tq = tmem + ((quad * 32u) << 16) + Cfg::kSf0;
        const uint32_t ready_leader = PAIR ? cluster_map(smem_u32(sf_ready), 0u) : 0u;
        Fp4Ring sr(prm.scale_stages), fr(Cfg::kSfSlots);
        bool ok = true;
        for (int t = cid; ok && t < tiles; t += ncl) {
            const int u1 = min(k1 * Cfg::kU, prm.units);
            for (int u = k0 * Cfg::kU; u < u1; ++u) {
                if (!fp4_warp_wait(&s_full[sr.slot], sr.phase, wd)) {
                    ok = false;
                    break;
                }
                const uint4 *sp = reinterpret_cast<const uint4 *>(scales + sr.slot * Cfg::kScaleStage);
                const uint4 *sq = sp + 128;
                uint32_t p[16], q[4 * Cfg::kQCols];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 v = sp[32 * j + lane];
                    p[j] = v.x;
                    p[4 + j] = v.y;
                    p[8 + j] = v.z;
                    p[12 + j] = v.w;
                }
#pragma unroll
                for (int j = 0; j < Cfg::kQCols; ++j) {
                    const uint4 v = 32 * j < BN ? sq[(32 * j + lane) & (BN - 1)] : make_uint4(0, 0, 0, 0);
                    q[j] = v.x;
                    q[Cfg::kQCols + j] = v.y;
                    q[2 * Cfg::kQCols + j] = v.z;
                    q[3 * Cfg::kQCols + j] = v.w;
                }
                fence_proxy_async_smem();  // generic reads before the TMA refills the stage
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[sr.slot]);
                sr.next();
                // padding bytes past the last block count as zero scales
                const int left = prm.k_blocks - 16 * u;
                if (left < 16) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) p[4 * w + j] = fp4_keep(p[4 * w + j], left - 4 * w);
#pragma unroll
                        for (int j = 0; j < Cfg::kQCols; ++j)
                            q[Cfg::kQCols * w + j] = fp4_keep(q[Cfg::kQCols * w + j], left - 4 * w);
                    }
                }
                if (!fp4_warp_wait(&sf_free[fr.slot], fr.phase ^ 1u, wd)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = tq + fr.slot * Cfg::kSfCols;
                tmem_st_32x32b_x16(at, p);
                if constexpr (Cfg::kQCols == 4)
                    tmem_st_32x32b_x16(at + 16, q);
                else
                    tmem_st_32x32b_x32(at + 16, q);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader)
                        mbar_arrive(&sf_ready[fr.slot]);
                    else
                        mbar_arrive_peer(ready_leader + 8u * static_cast<uint32_t>(fr.slot));
                }
                fr.next();
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int quad = warp;
        const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t empty_leader = PAIR ? cluster_map(smem_u32(acc_empty), 0u) : 0u;
        uint32_t nacc = 0;
        for (int t = cid; t < tiles; t += ncl, ++nacc) {
            const Fp4Tile x = fp4_tile<Cfg>(prm, first_tile, t, pr);
            const float alpha = prm.alpha ? __ldg(prm.alpha + x.e) : 1.0f;
            const uint32_t ab = nacc & 1u;
            const int n = x.p0 + quad * 32 + lane;
            const uint32_t tacc = trow + ab * Cfg::kAcc1;
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader)
                        mbar_arrive(&acc_empty[ab]);
                    else
                        mbar_arrive_peer(empty_leader + 8u * ab);
                }
            };
            if (!fp4_warp_wait(&acc_full[ab], (nacc >> 1) & 1u, wd)) break;
            tc_fence_after();
            if (cs > 1) {
                // split k: every CTA writes its partial of column group c / per to
                // CTA c / per, which adds them in rank order
                const int per = BN / cs, per_log2 = __ffs(per) - 1;  // cs is a power of two
                const uint32_t rb = nacc % Cfg::kRedBufs, rph = (nacc / Cfg::kRedBufs) & 1u;
                float *buf = red + rb * (BN * 128);
                if (!fp4_warp_wait_cluster(&red_empty[rb], rph ^ 1u, wd)) break;
#pragma unroll 1
                for (int c0 = 0; c0 < x.nq; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(tacc + c0, v);
                    tmem_ld_wait_regs(v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int c = c0 + j, owner = c >> per_log2;
                        st_cluster_u32(cluster_map(smem_u32(buf + (rank * per + (c & (per - 1))) * 128 + quad * 32 + lane),
                                                   static_cast<uint32_t>(owner)),
                                       v[j]);
                    }
                }
                release();
                if (lane < cs)
                    mbar_arrive_remote(cluster_map(smem_u32(&red_full[rb]), static_cast<uint32_t>(lane)));
                if (!fp4_warp_wait_cluster(&red_full[rb], rph, wd)) break;
                const int c1 = min(per, x.nq - rank * per);
                for (int c = 0; c < c1; ++c) {
                    float s = 0.0f;
                    for (int r = 0; r < cs; ++r) s += buf[(r * per + c) * 128 + quad * 32 + lane];
                    uint32_t v[1] = {__float_as_uint(s)};
                    fp4_store<1>(prm, v, alpha, static_cast<int64_t>(x.q0) + rank * per + c, 1, n);
                }
                __syncwarp();
                if (lane < cs)
                    mbar_arrive_remote(cluster_map(smem_u32(&red_empty[rb]), static_cast<uint32_t>(lane)));
                continue;
            }
            if constexpr (Cfg::kOverlap > 0) {
                // the columns that the other accumulator shares first, 96 at a time: once
                // they are in registers the next tile may start
                const int shared0 = ab ? 0 : BN - Cfg::kOverlap;
                uint32_t v[3][32];
#pragma unroll 1
                for (int c = shared0; c < shared0 + Cfg::kOverlap; c += 96) {
#pragma unroll
                    for (int i = 0; i < 3; ++i) tmem_ld_32x32b_x32(tacc + c + 32 * i, v[i]);
                    tmem_ld_wait_regs(v[0], v[1]);
                    tmem_ld_wait_regs(v[2]);
                    if (c + 96 == shared0 + Cfg::kOverlap) release();
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        fp4_store<32>(prm, v[i], alpha, static_cast<int64_t>(x.q0) + c + 32 * i, x.nq - c - 32 * i, n);
                }
                const int c_end = min(x.nq, ab ? BN : BN - Cfg::kOverlap);
#pragma unroll 1
                for (int c = ab ? Cfg::kOverlap : 0; c < c_end; c += 32) {
                    tmem_ld_32x32b_x32(tacc + c, v[0]);
                    tmem_ld_wait_regs(v[0]);
                    fp4_store<32>(prm, v[0], alpha, static_cast<int64_t>(x.q0) + c, c_end - c, n);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < x.nq; c += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(tacc + c, v);
                    tmem_ld_wait_regs(v);
                    fp4_store<16>(prm, v, alpha, static_cast<int64_t>(x.q0) + c, x.nq - c, n);
                }
                release();
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        if (leader && lane == 0) fp4_wait_drain(mma_drain, 0, prm.limit_ns);
        __syncwarp();
    }
    // no CTA of a cluster frees TMEM or leaves while another may still reach it
    if (csize > 1) cluster_sync_all();
    if (warp == 9) {
        tc_fence_after();
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem, Cfg::kTmemCols);
        else
            tmem_dealloc(tmem, Cfg::kTmemCols);
    }
}

}  // namespace igemm
