// Block-scaled fp8 GEMM, dense or grouped by expert:
//
//   C[m,n] = sum_kb sa[m,kb] sb[n/128,kb] sum_{k in block kb} a[m,k] b[n,k]
//
// with fp8 codes (both operands e4m3 or both e5m2), float32 scales per row and 128 k
// of A and per 128 x 128 tile of B, float32 accumulation.  The scales are any float32
// values, which the tensor core's own block scaling (powers of two) cannot take, so
// the tensor core writes a block's partial sums to one of PB buffers in tensor memory
// and the CUDA cores add it, times its scale, to totals in registers: 32 FMAs per
// output and 4096 k beside the MMAs, as f32x2 pairs.
//
// The weights B are the MMA's M side (128 rows per CTA) and the activations its N
// side, so that one kernel serves a single token (N = 16) and a prompt (N = 256 on a
// CTA pair) and the N of a ragged last tile is set per tile.  A scale then belongs to a
// column of the partial.  Loaded in fragment order (16x256b) a thread holds four
// rows of each of its columns, so that 16 bytes of scales serve 16 values; in the plain
// order (a lane a row) they would serve four, 1024 cycles of shared memory a block
// beside the 512 of its MMAs.
//
// CTA pairs turn tiles of more than 128 activations round (256 of them on the M side, 256
// weight rows on the N side): a lane's scale is then one number per block.
//
// Warps 0 .. EW-1 epilogue (four or eight), then two that issue MMAs (alternate blocks: a
// thread that waits after issuing resumes only when its MMAs are done; with one of them 16 x
// 28672 x 8192 39.7 us for 37.6), one that loads codes, one for the scales.  Persistent CTAs
// (or CTA pairs, or clusters that split k).  Every wait is bounded.
//
// What bounds it.  A few activations: HBM, the weights once (16 x 28672 x 8192: 37.7 to 38.3 us,
// 6.2 TB/s).  Many: the epilogue, which reads a block's 128 x 256 sums of each CTA from tensor
// memory and adds them in some 900 cycles, where the block's MMAs take 512 (8192^3: 427 to
// 460 us, 2390 to 2575 TFLOP/s at 1.7 to 2.0 GHz; the MMAs alone, without scales, 342 to
// 368 at 1.4 GHz and the part's power limit).
#pragma once
#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include "ptx.cuh"
#include "bsfp8.cuh"
#include "gemm_fp4_kernel.cuh"  // groups of rows, stores of a tile

namespace igemm {

struct Bsfp8Params {
    void *C;               // [rows, N] row-major
    int c_type;            // Fp4OutType
    const int *offsets;    // [experts + 1] rows of each group, or null: one group of all rows
    int rows, N, experts;
    int blocks;            // of 128 k: ceil(K / 128)
    int qt;                // activation rows per tile (Cfg::BN)
    int p_tiles;           // tiles of 128 weight rows (pair: of 256)
    int n_blocks;          // rows of scales per expert: ceil(N / 128)
    int group_p;           // tiles run in groups of group_p weight tiles (fastest) by every activation tile
    int cs;                // CTAs of a cluster that split k (1, 2 or 4)
    int slice;             // blocks of 128 k per CTA of such a cluster (a multiple of 4)
    int stream;            // single CTAs: the weights leave L2 first
    int format;            // 0 e4m3, 1 e5m2
    int stages;            // ring slots of codes
    int store_bytes;       // 16-bit C: bytes of a store (16, 4 or 2), as the alignment of its rows allows
    int wide;              // rows of C start on 32 bytes
    int off_scales, off_red, off_store, off_bars;  // shared-memory offsets after the code stages
    int *status;
    unsigned long long limit_ns;
    uint32_t limit_ns32;   // the same, at most 4 s
};

template <int BN_, bool PAIR_>
struct Bsfp8Cfg {
    static constexpr int BN = BN_;                     // most activation rows per tile
    static constexpr bool PAIR = PAIR_;
    static constexpr int CL = PAIR ? 2 : 1;
    // a block's partial sums are one accumulator of UN columns, or (pairs) two that are
    // multiplied, handed over and read apart
    static constexpr int kUnits = PAIR ? 2 : 1;
    static constexpr int UN = BN / kUnits;
    static constexpr int PB = 4;                       // accumulators in TMEM: blocks in turn
    static constexpr int kTurns = PB / kUnits;
    static constexpr int kParts = BN >= 64 ? 2 : 1;    // epilogue warps per TMEM lane quadrant
    static constexpr int CU = UN / kParts;             // most columns of an accumulator for each
    static constexpr int PC = kUnits * CU;             // ... of a tile
    static constexpr int EW = 4 * kParts;
    static constexpr int kQBox = BN / CL;              // activation rows this CTA loads
    // a tile with few activation rows loads them in one or two boxes of a quarter of the
    // full box
    static constexpr int kQRows = BN >= 128 ? kQBox / 4 : kQBox;
    static constexpr int kBoxP = 128 * 128;            // bytes of a block
    static constexpr int kBoxQ = kQBox * 128;
    static constexpr int kStage = kBoxP + kBoxQ;
    // four blocks' scales: BN rows of 16 bytes (turned: [4][BN]), then CL rows of the weights'
    static constexpr int kScaleStage = BN * 16 + 128;
    static constexpr int SS = PAIR ? 3 : BN == 128 ? 4 : 8;  // ring slots of scales
    static constexpr int kTmemCols = PB * UN;
    static constexpr int kRedBytes = BN <= 128 ? BN * 512 : 0;  // split k: the cluster's partials of this CTA's part
    static constexpr int kStoreBytes = EW * 2048;      // 16-bit C: 32 rows x 32 columns per epilogue warp
    // (16 activations: 166 KB of codes on their way to an SM; 16 x 28672 x 8192 with 8, 9, 10
    // and 11 slots 37.9, 37.6, 38.3 and 39.0 us)
    static constexpr int kMaxStages = BN == 16 ? 9 : 16;
    static constexpr int kNumBars = 2 * kMaxStages + 3 * SS + 2 * PB + 2 + 2 * EW;
    static constexpr int kBarBytes = (8 * kNumBars + 15) & ~15;
    static constexpr int kTailBytes = kBarBytes + 32;  // and the groups' table, 16 bytes each
    static constexpr int kWarpMma = EW, kWarpLoad = EW + 2, kWarpScale = EW + 3;
    static constexpr int kThreads = 32 * (EW + 4);
    static_assert(kStage % 1024 == 0 && kScaleStage % 128 == 0, "aligned operand tiles");
    static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM columns");
    static_assert(kTurns % 2 == 0, "an accumulator belongs to one of the two issuing warps");
    static_assert(!PAIR || BN == 256, "the pair form is built for 256 activation rows");
    static_assert(CU == 16 || CU == 32 || CU == 64, "whole loads");
    static_assert(EW * 8 * 16 <= kStoreBytes, "notices of a split k");

    // Whether a tile's activations are on the M side (144 to 224 of them through 8192 x 8192:
    // 34.7 us, 44.5 on the N side): then a block has two accumulators, else one.
    __device__ static bool lanes(int nq) { return PAIR && nq > UN; }
    // On the N side: columns of an accumulator that the epilogue's parts share evenly in 16s.
    __device__ static int columns(int nq) { return (nq + 16 * kParts - 1) / (16 * kParts) * (16 * kParts); }
};

// Tile t: group by binary search over the first tiles; whole tiles of qt activation rows
// and a remainder, in the grouped order of weight and activation tiles.
template <class Cfg>
__device__ __forceinline__ Fp4Tile bsfp8_tile(const Bsfp8Params &prm, const Fp4Group *groups, int t, int rank)
{
    int begin = 0, count = prm.rows, r = t, e = 0, q_tiles;
    if (prm.offsets) {
        int lo = 0, hi = prm.experts;  // groups[lo].x <= t, t below every later group's
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (groups[mid].x <= t) lo = mid;
            else hi = mid;
        }
        const Fp4Group g = groups[lo];
        e = lo;
        r = t - g.x;
        begin = g.y;
        count = g.z;
        q_tiles = g.w;
    } else {
        q_tiles = (count + prm.qt - 1) / prm.qt;
    }
    Fp4Tile x;
    x.e = e;
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

using F2 = float2;
__device__ __forceinline__ void bsfp8_fma2(F2 &t, uint32_t v0, uint32_t v1, F2 s)
{
    t = __ffma2_rn(make_float2(__uint_as_float(v0), __uint_as_float(v1)), s, t);
}
__device__ __forceinline__ uint32_t bsfp8_lo(F2 t) { return __float_as_uint(t.x); }
__device__ __forceinline__ uint32_t bsfp8_hi(F2 t) { return __float_as_uint(t.y); }
__device__ __forceinline__ F2 bsfp8_f2(float a, float b) { return make_float2(a, b); }
// 16 bytes of scales: the columns of 16 in the order of the fragments (columns 2 q, 2 q +
// 1, 8 + 2 q, 9 + 2 q at 4 q).
__device__ __forceinline__ int bsfp8_place(int column)
{
    return (column & ~15) + ((column >> 1) & 3) * 4 + ((column >> 3) & 1) * 2 + (column & 1);
}

template <int R>
__device__ __forceinline__ void bsfp8_regs_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void bsfp8_regs_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// fp4_warp_wait for the loop that sets the pace: by addresses, and the way taken when the
// barrier is not there yet needs few registers.
__device__ __forceinline__ uint32_t bsfp8_there(uint32_t bar, uint32_t parity)
{
    uint32_t there;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(there)
        : "r"(bar), "r"(parity)
        : "memory");
    return there;
}
__device__ __forceinline__ bool bsfp8_wait(uint32_t bar, uint32_t parity, uint32_t abort_at, const Bsfp8Params &prm)
{
    if (__all_sync(0xffffffffu, bsfp8_there(bar, parity))) return true;
    uint32_t start;  // (nanoseconds; 32 bits wrap after 4.3 s, and the limit is 4)
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(start));
#pragma unroll 1
    for (;;) {
        if (__all_sync(0xffffffffu, bsfp8_there(bar, parity))) return true;
        uint32_t now, aborted;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(aborted) : "r"(abort_at) : "memory");
        const bool late = now - start > prm.limit_ns32;
        if (__any_sync(0xffffffffu, late && !aborted)) {
            asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort_at), "r"(1) : "memory");
            atomicCAS(prm.status, 0, kStatusTimeout);
        }
        if (__any_sync(0xffffffffu, late || aborted)) return false;
    }
}

// Two barriers (their tests overlap when they are already complete).
__device__ __forceinline__ bool bsfp8_warp_wait2(uint64_t *a, uint32_t pa, uint64_t *b, uint32_t pb, const Watchdog &wd)
{
    const bool ra = mbar_try_wait(a, pa), rb = mbar_try_wait(b, pb);
    if (__all_sync(0xffffffffu, ra && rb)) return true;
    const bool ok = wait_bounded(a, pa, wd) && wait_bounded(b, pb, wd);
    return __all_sync(0xffffffffu, ok);
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    igemm_bsfp8_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                       const __grid_constant__ CUtensorMap mapQs, const __grid_constant__ CUtensorMap mapSP,
                       const __grid_constant__ CUtensorMap mapSQ, const Bsfp8Params prm)
{
    constexpr bool PAIR = Cfg::PAIR;
    constexpr int BN = Cfg::BN, PB = Cfg::PB, SS = Cfg::SS, EW = Cfg::EW, CU = Cfg::CU, PC = Cfg::PC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *codes = smem;
    uint8_t *scales = smem + prm.off_scales;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + prm.off_bars);
    uint64_t *full = bars;                        // [stages] codes landed (pair: both CTAs', in the even CTA)
    uint64_t *empty = full + Cfg::kMaxStages;     // [stages] consumed (MMA commit), and seen by the other issuing warp
    uint64_t *s_raw = empty + Cfg::kMaxStages;    // [SS] scale rows landed
    uint64_t *s_full = s_raw + SS;                // [SS] ... turned (scale warp)
    uint64_t *s_empty = s_full + SS;              // [SS] read (epilogue warps)
    uint64_t *p_full = s_empty + SS;              // [PB] an accumulator complete (commit)
    uint64_t *p_empty = p_full + PB;              // [PB] ... read by the epilogue warps (pair: both CTAs', in the even CTA)
    uint64_t *mma_drain = p_empty + PB;           // [2]
    uint64_t *red_full = mma_drain + 2;           // [EW] split k: the other CTAs' partials for this warp landed
    uint64_t *red_empty = red_full + EW;          // [EW] ... and the other CTAs have read what this warp sent
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + prm.off_bars + Cfg::kBarBytes);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *total_slot = reinterpret_cast<int *>(tmem_slot + 2);
    uint8_t *fixed = reinterpret_cast<uint8_t *>(tmem_slot) + 16;  // 16 bytes that stay as they are
    Fp4Group *groups = reinterpret_cast<Fp4Group *>(smem + prm.off_bars + Cfg::kTailBytes);
    // split k: 16 bytes for each notice of another CTA, never read ([EW][4 CTAs], in the
    // staging of stores, which it does not use)
    uint8_t *notices = smem + prm.off_store;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int cs = PAIR ? 1 : prm.cs;
    const int csize = PAIR ? 2 : cs;
    const int rank = csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int pr = PAIR ? rank : 0;  // half of the pair's tile
    const int cid = blockIdx.x / csize, ncl = gridDim.x / csize;
    const bool leader = !PAIR || rank == 0;

    if (warp == Cfg::kWarpLoad) {
        if (lane < prm.stages) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 2);
        }
        if (lane < SS) {
            mbar_init(&s_raw[lane], 1);
            mbar_init(&s_full[lane], 1);
            mbar_init(&s_empty[lane], EW);
        }
        if (lane < PB) {
            mbar_init(&p_full[lane], 1);
            mbar_init(&p_empty[lane], EW * Cfg::CL);
        }
        if (lane < 2) mbar_init(&mma_drain[lane], 1);
        if (cs > 1 && lane < EW) {
            mbar_init(&red_full[lane], 1);
            mbar_init(&red_empty[lane], 1);
        }
        if (lane == 0) {
            *abort_flag = 0;
            tma_prefetch_map(&mapP);
            tma_prefetch_map(&mapQ);
            if (Cfg::kQRows < Cfg::kQBox) tma_prefetch_map(&mapQs);
            tma_prefetch_map(&mapSP);
            tma_prefetch_map(&mapSQ);
        }
        fence_mbar_init();
    }
    if (warp == Cfg::kWarpMma) {
        if constexpr (PAIR) {
            tmem_alloc_pair(tmem_slot, Cfg::kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, Cfg::kTmemCols);
            tmem_relinquish();
        }
    }
    if (warp == 0) {
        if (prm.offsets) {
            // running tile counts of the groups (the offsets may come from the kernel before)
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int run = 0;
            for (int e0 = 0; e0 < prm.experts; e0 += 32) {
                const Fp4Group g = fp4_groups32(prm, e0, run);
                if (e0 + lane < prm.experts) groups[e0 + lane] = g;
            }
            if (lane == 0) *total_slot = run;
        } else if (lane == 0) {
            *total_slot = (prm.rows + prm.qt - 1) / prm.qt * prm.p_tiles;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tiles = *total_slot;
    if (csize > 1) cluster_sync_all();  // the other CTAs' barriers are initialised
    // Up to here the kernel before this one in the stream may still run.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Watchdog wd{abort_flag, prm.status, prm.limit_ns};
    // this CTA's slice of k, in blocks (split k: the cluster rank's)
    const int b0 = PAIR ? 0 : min(rank * prm.slice, prm.blocks);
    const int b1 = PAIR ? prm.blocks : min(b0 + prm.slice, prm.blocks);

    if (warp >= EW) {
        // (of 168 registers a thread at the launch: 256 x 224 + 128 x 56 = 384 x 168)
        if constexpr (PAIR) bsfp8_regs_dec<56>();
        if (warp == Cfg::kWarpLoad) {
            // -------------------------------------------------------- codes
            Fp4Ring cr(prm.stages);
            const bool stream = !PAIR && prm.stream;
            const uint64_t evict_first = l2_policy_evict_first();
            uint32_t issued = 0, last = 0;
            bool ok = true;
            for (int t = cid; ok && t < tiles; t += ncl) {
                const Fp4Tile x = bsfp8_tile<Cfg>(prm, groups, t, pr);
                // activation rows that this CTA loads (pair: half of the tile's)
                const int mine = !PAIR ? x.nq : Cfg::lanes(x.nq) ? 128 : Cfg::columns(x.nq) / 2;
                const bool small = Cfg::kQRows < Cfg::kQBox && mine <= 2 * Cfg::kQRows;
                const bool two = small && mine > Cfg::kQRows;
                const int py = x.e * prm.N + x.p0, qy = x.q0 + pr * mine;
                const uint32_t tx = static_cast<uint32_t>(Cfg::kBoxP +
                                                          (!small ? Cfg::kBoxQ : (two ? 2 : 1) * Cfg::kQRows * 128));
                const CUtensorMap *mq = small ? &mapQs : &mapQ;
#pragma unroll 1
                for (int b = b0; b < b1; ++b) {
                    if (!fp4_warp_wait(&empty[cr.slot], cr.phase ^ 1u, wd)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t *to = codes + cr.slot * Cfg::kStage, *tq = to + Cfg::kBoxP;
                        if constexpr (PAIR) {
                            // both CTAs' bytes count on the even CTA's barrier
                            if (leader) mbar_arrive_expect_tx(&full[cr.slot], 2 * tx);
                            const uint32_t bar = cluster_map(smem_u32(&full[cr.slot]), 0u);
                            tma_load_2d_pair(to, &mapP, bar, b * 128, py);
                            tma_load_2d_pair(tq, mq, bar, b * 128, qy);
                            if (two) tma_load_2d_pair(tq + Cfg::kQRows * 128, mq, bar, b * 128, qy + Cfg::kQRows);
                        } else {
                            mbar_arrive_expect_tx(&full[cr.slot], tx);
                            if (stream) tma_load_2d_hint(to, &mapP, &full[cr.slot], b * 128, py, evict_first);
                            else tma_load_2d(to, &mapP, &full[cr.slot], b * 128, py);
                            tma_load_2d(tq, mq, &full[cr.slot], b * 128, qy);
                            if (two) tma_load_2d(tq + Cfg::kQRows * 128, mq, &full[cr.slot], b * 128, qy + Cfg::kQRows);
                        }
                    }
                    __syncwarp();
                    issued |= 1u << cr.slot;
                    last = (last & ~(1u << cr.slot)) | (cr.phase << cr.slot);
                    cr.next();
                }
            }
            // never leave with copies in flight, nor with an MMA commit on its way here
            const uint64_t t0 = globaltimer_ns();
            if (leader) fp4_drain(full, issued, last, t0, prm.limit_ns);
            fp4_drain(empty, issued, last, t0, prm.limit_ns);
        } else if (warp == Cfg::kWarpScale) {
            // -------------------------------------------------------- scales
            // Four blocks at a time.  The loads run SS - 1 groups of blocks ahead of the
            // turning, so that the slot of the next one is that of the group before, which
            // the epilogue leaves while it has the turned one still to do.
            Fp4Ring lr(SS), sr(SS);
            uint32_t issued = 0, last = 0;
            bool ok = true;
            int lt = cid, lb = b0;  // next to load
            const auto load = [&] {
                const Fp4Tile x = bsfp8_tile<Cfg>(prm, groups, lt, pr);
                ok = fp4_warp_wait(&s_empty[lr.slot], lr.phase ^ 1u, wd);
                if (!ok) return;
                fence_proxy_async_smem();  // this warp's earlier writes of turned scales come before the copies
                __syncwarp();
                if (elect_one()) {
                    uint8_t *to = scales + lr.slot * Cfg::kScaleStage;
                    mbar_arrive_expect_tx(&s_raw[lr.slot], BN * 16 + Cfg::CL * 16);
                    tma_load_2d(to, &mapSQ, &s_raw[lr.slot], lb * 4, x.q0);
                    tma_load_2d(to + BN * 16, &mapSP, &s_raw[lr.slot], lb * 4,
                                x.e * prm.n_blocks + (x.p0 / 128 - pr));
                }
                __syncwarp();
                issued |= 1u << lr.slot;
                last = (last & ~(1u << lr.slot)) | (lr.phase << lr.slot);
                lr.next();
                lb += 4;
                if (lb >= b1) {
                    lb = b0;
                    lt += ncl;
                }
            };
            if (b0 < b1) {
                for (int i = 0; i < SS - 1 && ok && lt < tiles; ++i) load();
                for (int t = cid; ok && t < tiles; t += ncl) {
                    const Fp4Tile x = bsfp8_tile<Cfg>(prm, groups, t, pr);
                    const bool lanes = Cfg::lanes(x.nq);
                    for (int b = b0; ok && b < b1; b += 4) {
                        ok = fp4_warp_wait(&s_raw[sr.slot], sr.phase, wd);
                        if (!ok) break;
                        if (!lanes) {
                            // [BN][4] to [4][BN], times the weights' scale
                            float4 *raw = reinterpret_cast<float4 *>(scales + sr.slot * Cfg::kScaleStage);
                            float *to = reinterpret_cast<float *>(raw);
                            const float4 sb = raw[BN + pr];
                            constexpr int R = (BN + 31) / 32;
                            float4 v[R];
#pragma unroll
                            for (int i = 0; i < R; ++i)
                                if (32 * i + lane < BN) v[i] = raw[32 * i + lane];
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < R; ++i)
                                if (32 * i + lane < BN) {
                                    const int at = bsfp8_place(32 * i + lane);
                                    to[at] = v[i].x * sb.x;
                                    to[BN + at] = v[i].y * sb.y;
                                    to[2 * BN + at] = v[i].z * sb.z;
                                    to[3 * BN + at] = v[i].w * sb.w;
                                }
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_full[sr.slot]);
                        sr.next();
                        if (lt < tiles) load();
                    }
                }
            }
            const uint64_t t0 = globaltimer_ns();
            fp4_drain(s_raw, issued, last, t0, prm.limit_ns);
        } else if (leader) {
            // -------------------------------------------------------- MMA issuers
            // A block each in turn; of a pair's tile with two accumulators, one of every block
            // each (an accumulator always belongs to the same warp).
            const int me = warp - Cfg::kWarpMma;
            const uint64_t desc0 = sdesc_kmajor_sw128(smem_u32(codes));
            const uint32_t fmt = static_cast<uint32_t>(prm.format);
            Fp4Ring cr(prm.stages);
            uint32_t phases = 0;  // of the accumulators
            bool ok = true;
            for (int t = cid; ok && t < tiles; t += ncl) {
                const Fp4Tile x = bsfp8_tile<Cfg>(prm, groups, t, pr);
                const bool lanes = Cfg::lanes(x.nq);
                const int cols = lanes ? Cfg::UN : Cfg::columns(x.nq);
                const uint32_t idesc = idesc_f8_f32(128 * Cfg::CL, static_cast<uint32_t>(cols), fmt);
                // the second accumulator: the other half of each CTA's rows on the N side
                const uint64_t half = lanes ? static_cast<uint64_t>(me * (64 * 128 >> 4)) : 0;
                for (int b = b0; b < b1; ++b) {
                    const bool mine = lanes || (b & 1) == me;
                    const uint32_t pb = lanes ? 2 * (b & 1) + me : b % PB;
                    if (!mine) {
                        // The slot's other arrival, in its turn: both warps see every use of a slot, so
                        // that a wait by parity is never passed by the use before.
                        ok = fp4_warp_wait(&full[cr.slot], cr.phase, wd);
                        if (!ok) break;
                        if (elect_one()) {
                            if constexpr (PAIR) mma_commit_pair_multicast(&empty[cr.slot], 0x3);
                            else mbar_arrive(&empty[cr.slot]);
                        }
                        __syncwarp();
                    }
                    if (mine) {
                        const uint32_t phase = phases >> pb & 1u;
                        phases ^= 1u << pb;
                        if (!bsfp8_warp_wait2(&p_empty[pb], phase ^ 1u, &full[cr.slot], cr.phase, wd)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t p0 = desc0 + static_cast<uint64_t>(cr.slot * (Cfg::kStage >> 4));
                            const uint64_t q0 = p0 + static_cast<uint64_t>(Cfg::kBoxP >> 4);
                            const uint64_t da = lanes ? q0 : p0, db = (lanes ? p0 : q0) + half;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if constexpr (PAIR)
                                    mma_f8f6f4_pair(tmem + pb * Cfg::UN, da + 2 * q, db + 2 * q, idesc, q > 0 ? 1u : 0u);
                                else
                                    mma_f8f6f4(tmem + pb * Cfg::UN, da + 2 * q, db + 2 * q, idesc, q > 0 ? 1u : 0u);
                            }
                            if constexpr (PAIR) {
                                mma_commit_pair_multicast(&p_full[pb], 0x3);
                                mma_commit_pair_multicast(&empty[cr.slot], 0x3);
                            } else {
                                mma_commit(&p_full[pb]);
                                mma_commit(&empty[cr.slot]);
                            }
                        }
                        __syncwarp();
                    }
                    cr.next();
                }
            }
            if (elect_one()) {
                if constexpr (PAIR) mma_commit_pair(&mma_drain[me]);
                else mma_commit(&mma_drain[me]);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ epilogue
        if constexpr (PAIR) bsfp8_regs_inc<224>();
        const int quad = warp & 3, part = warp >> 2;
        const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        uint8_t *stage = smem + prm.off_store + warp * 2048;
        // (the even CTA's; single CTAs: their own)
        const uint32_t empty_leader = csize > 1 ? cluster_map(smem_u32(p_empty), PAIR ? 0u : rank) : smem_u32(p_empty);
        const uint32_t abort_at = smem_u32(const_cast<int *>(abort_flag)), p_full_at = smem_u32(p_full), s_full_at = smem_u32(s_full);
        const int q4 = lane & 3;
        Fp4Ring sr(SS);
        uint32_t phases = 0;         // of the accumulators
        uint32_t n = 0, armed = 0;  // armed: split k, tiles whose partials this warp expects
        bool ok = true;
        for (int t = cid; t < tiles; t += ncl, ++n) {
            const Fp4Tile x = bsfp8_tile<Cfg>(prm, groups, t, pr);
            const bool lanes = Cfg::lanes(x.nq);
            // this warp's columns of an accumulator (activations on the N side: of the tile)
            const int cu = (lanes ? Cfg::UN : Cfg::columns(x.nq)) / Cfg::kParts, c0 = part * cu;
            const int cols = min(x.nq - c0, cu);
            const uint32_t tpart = trow + part * cu;
            // The blocks of the tile, an accumulator at a time: load(address, to) brings all its
            // columns of this warp to registers, it is released, and add(begin(scales, block),
            // h, from) adds them, while the other warp of the SM's quarter loads.  (A CTA that
            // gives up runs on without waiting: an exit costs registers and moves.)
            const auto blocks = [&](auto units, auto load, auto begin, auto add) {
                constexpr int count = decltype(units)::value;
                const auto block = [&](const float *slot, int j) {
                    const auto sc = begin(slot, j);
                    bool early = false;
#pragma unroll
                    for (int h = 0; h < count; ++h) {
                        const uint32_t pb = count == 2 ? 2 * (j & 1) + h : j % PB, phase = phases >> pb & 1u;
                        if (h == 0 || !early) ok &= bsfp8_wait(p_full_at + 8 * pb, phase, abort_at, prm);
                        tc_fence_after();
                        phases ^= 1u << pb;
                        uint32_t v[CU];
                        load(tpart + pb * Cfg::UN, v);
                        // (the next one's test is on its way meanwhile)
                        if (h + 1 < count) early = bsfp8_there(p_full_at + 8 * (pb + 1), phases >> (pb + 1) & 1u);
                        tmem_ld_wait_regs(v);
                        tc_fence_before();
                        if (lane == 0) mbar_arrive_peer(empty_leader + 8 * pb);
                        add(sc, h, v);
                        if (h + 1 < count) early = __all_sync(0xffffffffu, early);
                    }
                };
#pragma unroll 1
                for (int b = b0; b < b1; b += 4) {
                    ok &= bsfp8_wait(s_full_at + 8 * sr.slot, sr.phase, abort_at, prm);
                    const float *slot = reinterpret_cast<const float *>(scales + sr.slot * Cfg::kScaleStage);
                    const int some = min(4, b1 - b);
#pragma unroll 1
                    for (int j = 0; j < some; j += 2) {
                        block(slot, j);
                        if (j + 1 < some) block(slot, j + 1);
                    }
                    __syncwarp();  // (read; what the scale warp wrote there it orders before its copies itself)
                    if (lane == 0) mbar_arrive(&s_empty[sr.slot]);
                    sr.next();
                }
            };
            if constexpr (PAIR) if (lanes) {
                // a lane an activation row, the part's columns one block of weight rows
                F2 tot[PC / 2];
#pragma unroll
                for (int i = 0; i < PC / 2; ++i) tot[i] = make_float2(0.0f, 0.0f);
                const auto load = [&](uint32_t at, uint32_t(&to)[CU]) { tmem_ld_32x32b_x64(at, to); };
                const auto begin = [&](const float *sc, int kb) {
                    const float s = sc[(rank * 128 + quad * 32 + lane) * 4 + kb] * sc[(BN + part) * 4 + kb];
                    return bsfp8_f2(s, s);
                };
                const auto add = [&](F2 ss, int h, const uint32_t(&w)[CU]) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) bsfp8_fma2(tot[h * (CU / 2) + j], w[2 * j], w[2 * j + 1], ss);
                };
                blocks(std::integral_constant<int, 2>(), load, begin, add);
                if (!ok) break;
                // A lane's row of 128 columns, 16 words at a time: as two stores of 32 bytes, or,
                // where rows of C start elsewhere, through shared memory (64-byte rows, 16-byte
                // chunk c of row r at c ^ (r / 2 % 4)) to leave as 64 contiguous bytes of two rows.
                const int nb = x.p0 - 128 * pr + part * 128, r0 = rank * 128 + quad * 32;
                const bool f32 = prm.c_type == kOutF32, bf16 = prm.c_type == kOutBf16;
                const int row_words = f32 ? prm.N : prm.N / 2;  // (N is even)
                const int64_t at = (static_cast<int64_t>(x.q0) + r0) * row_words + (f32 ? nb : nb / 2);
                uint32_t *to = static_cast<uint32_t *>(prm.C) + at;
                const int left = row_words - (f32 ? nb : nb / 2), rows = x.nq - r0;
                const auto leave = [&](int word, const uint32_t(&w)[16]) {
                    if (word >= left) return;  // (the same in every lane)
                    if (prm.wide) {
                        if (lane < rows) {
                            uint32_t *from = to + static_cast<int64_t>(lane) * row_words + word;
                            st_v8(from, reinterpret_cast<const uint32_t(&)[8]>(w[0]));
                            if (word + 8 < left) st_v8(from + 8, reinterpret_cast<const uint32_t(&)[8]>(w[8]));
                        }
                        return;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4 *>(stage + lane * 64 + ((q ^ (lane >> 1 & 3)) << 4)) =
                            make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
                    __syncwarp();
                    const int c = lane & 15;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int r = 2 * i + (lane >> 4);
                        const uint32_t v = *reinterpret_cast<const uint32_t *>(
                            stage + r * 64 + (((c >> 2) ^ (r >> 1 & 3)) << 4) + (c & 3) * 4);
                        if (r < rows && word + c < left) to[static_cast<int64_t>(r) * row_words + word + c] = v;
                    }
                    __syncwarp();  // read before the next words overwrite them
                };
                if (f32) {
#pragma unroll
                    for (int j = 0; j < PC; j += 16) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            w[2 * i] = bsfp8_lo(tot[j / 2 + i]);
                            w[2 * i + 1] = bsfp8_hi(tot[j / 2 + i]);
                        }
                        leave(j, w);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < PC / 2; j += 16) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            if (bf16) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(tot[j + i].x, tot[j + i].y);
                                w[i] = *reinterpret_cast<const uint32_t *>(&h);
                            } else {
                                const __half2 h = __floats2half2_rn(tot[j + i].x, tot[j + i].y);
                                w[i] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                        }
                        leave(j, w);
                    }
                }
                continue;
            }
            // 16 columns of fragments at a time.  Pairs of totals: 16 columns (8 i), lanes
            // 0-15 and 16-31 (4 e), column octet (2 j), row octet (o).
            F2 tot[CU / 2];
#pragma unroll
            for (int i = 0; i < CU / 2; ++i) tot[i] = make_float2(0.0f, 0.0f);
            const auto load = [&](uint32_t at, uint32_t(&to)[CU]) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t from = at + (static_cast<uint32_t>(16 * e) << 16);
                    if constexpr (CU == 64) tmem_ld_16x256b_x8(from, to + e * (CU / 2));
                    else if constexpr (CU == 32) tmem_ld_16x256b_x4(from, to + e * (CU / 2));
                    else tmem_ld_16x256b_x2(from, to + e * (CU / 2));
                }
            };
            // (read before the wait for the partial sums)
            struct Scales {
                float4 of[CU / 16];
            };
            const auto begin = [&](const float *sc, int kb) {
                Scales s;
                const float *from = sc + kb * BN + c0 + 4 * q4;
#pragma unroll
                for (int c = 0; c < CU / 16; ++c) s.of[c] = *reinterpret_cast<const float4 *>(from + 16 * c);
                return s;
            };
            const auto add = [&](const Scales &sc, int, const uint32_t(&v)[CU]) {
#pragma unroll
                for (int c = 0; c < CU / 16; ++c) {
                    const float4 s = sc.of[c];
                    const F2 s01 = bsfp8_f2(s.x, s.y), s23 = bsfp8_f2(s.z, s.w);
                    F2 *to = tot + 8 * c;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            const int at = e * (CU / 2) + 8 * c + 2 * o;
                            bsfp8_fma2(to[4 * e + o], v[at], v[at + 1], s01);
                            bsfp8_fma2(to[4 * e + 2 + o], v[at + 4], v[at + 5], s23);
                        }
                }
            };
            blocks(std::integral_constant<int, 1>(), load, begin, add);
            if (!ok) break;
            const int n0 = x.p0 + quad * 32;
            if (cs > 1) {
                // split k: CTA r adds the parts of row octets r .. of the cluster's CTAs in
                // rank order (fixed, whatever arrives first).  An octet's 16 columns are 16
                // bytes a lane, at [sender][warp][(16 columns, octet of the owner)][lane].
                const int per = 4 / cs;               // octets of an owner
                constexpr int C16 = CU / 16;
                const int units = C16 * per;
                uint4 *buf = reinterpret_cast<uint4 *>(smem + prm.off_red) + lane;
                const uint32_t ph = n & 1u;
                if (lane == 0) mbar_arrive_expect_tx(&red_full[warp], static_cast<uint32_t>((cs - 1) * units * 512));
                ++armed;
                ok = fp4_warp_wait_cluster(&red_empty[warp], ph ^ 1u, wd);
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < C16; ++c)
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        const int owner = o / per;
                        const F2 *from = tot + 8 * c + 4 * (o >> 1) + (o & 1);
                        const uint32_t v[4] = {bsfp8_lo(from[0]), bsfp8_hi(from[0]), bsfp8_lo(from[2]), bsfp8_hi(from[2])};
                        if (owner != rank) {
                            const uint4 *to = buf + ((rank * EW + warp) * units + c * per + o % per) * 32;
                            st_async_v4(cluster_map(smem_u32(to), static_cast<uint32_t>(owner)), v,
                                        cluster_map(smem_u32(&red_full[warp]), static_cast<uint32_t>(owner)));
                        }
                    }
                ok = fp4_warp_wait_cluster(&red_full[warp], ph, wd);
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < C16; ++c)
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        if (o / per != rank) continue;
                        const F2 *own = tot + 8 * c + 4 * (o >> 1) + (o & 1);
                        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        for (int r = 0; r < cs; ++r) {
                            const uint4 v = r == rank ? make_uint4(bsfp8_lo(own[0]), bsfp8_hi(own[0]), bsfp8_lo(own[2]),
                                                                   bsfp8_hi(own[2]))
                                                      : buf[((r * EW + warp) * units + c * per + o % per) * 32];
                            s[0] += __uint_as_float(v.x);
                            s[1] += __uint_as_float(v.y);
                            s[2] += __uint_as_float(v.z);
                            s[3] += __uint_as_float(v.w);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int col = 16 * c + 8 * (j >> 1) + 2 * q4 + (j & 1);
                            if (col < cols)
                                fp4_store1(prm, s[j], static_cast<int64_t>(x.q0) + c0 + col,
                                           n0 + 8 * o + (lane >> 2));
                        }
                    }
                __syncwarp();
                // read: the other CTAs may write again, where a later tile does.  Each is sent
                // 16 bytes (no matter which): this warp's reads come before that copy, so before
                // its completion, a release at cluster scope.
                if (t + ncl < tiles) {
                    if (lane == 0) mbar_arrive_expect_tx(&red_empty[warp], 16u * (cs - 1));
                    if (lane < cs && lane != rank)
                        bulk_copy_to_cta(cluster_map(smem_u32(notices + 16 * (4 * warp + rank)), lane), fixed, 16,
                                         cluster_map(smem_u32(&red_empty[warp]), lane));
                }
                continue;
            }
            if (prm.c_type == kOutF32) {
                // (a store: eight columns of C of each of four rows)
                float *to = static_cast<float *>(prm.C) + (static_cast<int64_t>(x.q0) + c0 + 2 * q4) * prm.N + n0 +
                            (lane >> 2);
#pragma unroll
                for (int c = 0; c < CU / 8; ++c) {
                    const int col = 8 * c;
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        const F2 v = tot[8 * (c >> 1) + 4 * (o >> 1) + 2 * (c & 1) + (o & 1)];
                        if (n0 + 8 * o + (lane >> 2) < prm.N) {
                            float *at = to + static_cast<int64_t>(col) * prm.N + 8 * o;
                            if (col + 2 * q4 < cols) at[0] = __uint_as_float(bsfp8_lo(v));
                            if (col + 2 * q4 + 1 < cols) at[prm.N] = __uint_as_float(bsfp8_hi(v));
                        }
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < CU; c += 32) {
                    if (c < cols) {
                        uint32_t v[2][16];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                // (fragments: lanes 0-15 and 16-31, column octet, row octet)
                                const int from = c / 2 + 8 * i + j;
                                const bool there = c + 16 * i < CU;
                                const F2 w = there ? tot[there ? from : 0] : make_float2(0.0f, 0.0f);
                                v[i][2 * j] = bsfp8_lo(w);
                                v[i][2 * j + 1] = bsfp8_hi(w);
                            }
                        fp4_store32_cols<false>(prm, v, 1.0f, static_cast<int64_t>(x.q0) + c0 + c, cols - c, n0, stage);
                    }
                }
            }
        }
        // gave up: another CTA's partials may be on their way here, and its notices
        if (cs > 1 && !ok) {
            const uint64_t t0 = globaltimer_ns();
            const auto drain = [&](uint64_t *bar, uint32_t parity) {
                while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < prm.limit_ns) {
                }
            };
            if (n > 0) drain(&red_empty[warp], (n - 1) & 1u);
            if (lane == 0 && n >= armed)
                mbar_arrive_expect_tx(&red_full[warp], static_cast<uint32_t>((cs - 1) * (CU / 16) * (4 / cs) * 512));
            drain(&red_full[warp], n & 1u);
        }
    }

    // ---------------------------------------------------------------- teardown
    // The next kernel may be set up on SMs that this one has left; it waits for the end
    // of this grid before it touches memory.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (warp == Cfg::kWarpMma) {
        if (leader && lane == 0) fp4_drain(mma_drain, 3u, 0u, globaltimer_ns(), prm.limit_ns);
        __syncwarp();
    }
    // no CTA of a cluster frees TMEM or leaves while another may still reach it
    if (csize > 1) cluster_sync_all();
    if (warp == Cfg::kWarpMma) {
        tc_fence_after();
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem, Cfg::kTmemCols);
        else
            tmem_dealloc(tmem, Cfg::kTmemCols);
    }
}

}  // namespace igemm
