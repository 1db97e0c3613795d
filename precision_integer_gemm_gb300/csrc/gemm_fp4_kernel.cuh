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
// A block of 512 k is the unit of the loop: two stages of codes (256 k, 128 bytes a
// row, each with its own slot) and the block's scales.  These stay row-major as
// the caller has them, 16 (mx) or 32 (nv) bytes a row and block, at any row (a
// group starts anywhere).  The tensor core wants the words (4 bytes) of 128 rows
// across 4 columns of all four TMEM lane quadrants.  A block's rows land in a
// small ring by TMA, in order with the codes; a warp per 128 rows turns them in
// place (lane i reads rows i, 32 + i, 64 + i, 96 + i and writes word w of the four as 16
// bytes of the w-th 512), and tcgen05.cp spreads the 512s over the quadrants, in
// order with the MMAs.  So scales cost four times their bytes in shared-memory
// traffic beside the codes' 32 KB written and read per stage.
// (Loaded with plain loads, the scales waited microseconds behind the operand
// stream: 338 us at 8192^3.  Stored to TMEM by a warp per quadrant, every scale
// was read four times.)
//
// What a single warp issues sets the pace of the loop: an MMA takes it about 50
// cycles, a TMA load 100, a successful wait 50 to 100, and a block's MMAs run for
// 1024.  So a block has one joint wait for its 8 MMAs, and weights, activations and
// scales each have a loading warp (one warp for all three took 1500 cycles a block).
//
// Few rows are bound by HBM: 16 x 28672 x 8192 nv takes 21.5 us, 6.2 TB/s (launch, first
// stage and tail beside it).  Many rows are bound by the tensor core and its operands:
// 8192^3 mx takes 155 us alone, 7.1 PFLOP/s, 1200 cycles a block where the MMAs take
// 1024; back to back the power cap makes it 171 to 176 us.
//
// Warps 0-3 epilogue, 4 MMA issue, 5 weight loads, 6 activation loads, 7 scale loads,
// 8 and up scales.  Persistent CTAs (or CTA pairs, or clusters that split k).  Every
// wait is bounded.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "ptx.cuh"

namespace igemm {

constexpr int kFp4MaxExperts = 1024;
constexpr int kFp4MaxTiles = 0x3FFFFFFF;  // of one call

enum Fp4OutType : int { kOutF32 = 0, kOutBf16 = 1, kOutF16 = 2 };

struct Fp4Params {
    void *C;               // [rows, N] row-major
    int c_type;            // Fp4OutType
    const float *alpha;    // [experts] or null (1)
    const int *offsets;    // [experts + 1] rows of each group, or null: one group of all rows
    int rows, N, experts;
    int k_steps;           // MMA steps of 64 k: ceil(K / 64)
    int k_blocks;          // scale bytes in use per row
    int blocks;            // of 512 k: ceil(K / 512)
    int qt;                // activation rows per tile (<= BN)
    int p_tiles;           // tiles of 128 weight rows (pair: of 256)
    int group_p;           // tiles run in groups of group_p weight tiles (fastest) by every activation tile
    int cs;                // CTAs of a cluster that split k (1: none; a power of two, 4 cs <= BN)
    int blocks_per_slice;
    int stream;            // single CTAs: the weights leave L2 first
    int prefetch;          // single CTAs: stages of weights that go to L2 ahead of the kernel's turn
    int code_stages, scale_stages;  // ring slots: 256 k of codes, 512 k of scales
    int store_bytes;       // 16-bit C: bytes of a store (16, 4 or 2), as the alignment of its rows allows
    int off_scales, off_red, off_store, off_bars;  // shared-memory offsets after the code stages
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
    static constexpr int kH = NV ? 2 : 1;              // 16-byte pieces of a row's scales per block
    static constexpr int kBoxP = 128 * 128;            // bytes of 256 k
    static constexpr int kBoxQ = kQBox * 128;
    // a tile with few activation rows loads them in one or two boxes of a quarter of
    // the full box (four of them for every tile measured 205 against 182 us at
    // 8192^3)
    static constexpr int kQRows = BN >= 128 ? kQBox / 4 : kQBox;
    static constexpr int kStage = kBoxP + kBoxQ;
    static constexpr int kQGroups = (BN + 127) / 128;  // groups of 128 activation rows
    static constexpr int kQScaleRows = BN < 128 ? BN : 128;  // rows of a scale box of the activations
    static constexpr int kGroupBytes = kH * 2048;            // a block's scales of 128 rows
    static constexpr int kScaleStage = (1 + kQGroups) * kGroupBytes;
    static constexpr int kMaxScaleStages = 4;
    static constexpr int kQCols = BN <= 128 ? 4 : BN / 32;   // TMEM columns of one word of every activation row
    static constexpr int kSfCols = 16 + 4 * kQCols;    // TMEM columns of four words: a block (mx), a stage (nv)
    static constexpr int kSfSlots = 2;                 // such sets of columns, used in turn
    // two accumulators of BN columns; with BN = 256 the second starts before
    // the first ends (kOverlap columns), so that the scales fit beside them
    static constexpr int kAcc1 = BN == 256 ? 512 - kSfSlots * kSfCols - BN : BN;
    static constexpr int kOverlap = BN - kAcc1;
    static constexpr int kSf0 = kAcc1 + BN;
    static constexpr int kTmemUse = kSf0 + kSfSlots * kSfCols;
    static constexpr int kTmemCols = kTmemUse <= 128 ? 128 : kTmemUse <= 256 ? 256 : 512;
    static constexpr int kRedBufs = BN <= 32 ? 2 : 1;
    static constexpr int kRedBytes = kRedBufs * BN * 512;  // split k (BN <= 64): partial tiles of the cluster's CTAs
    static constexpr int kMaxStages = 16;
    static constexpr int kNumBars = 2 * kMaxStages + 3 * kMaxScaleStages + 4 + 1 + 16;
    static constexpr int kStoreBytes = 4 * 2048;  // 16-bit C: 32 rows x 32 columns per epilogue warp
    static constexpr int kNoticeBytes = PAIR ? 16 * kMaxScaleStages : 0;
    static constexpr int kTailBytes = 8 * kNumBars + 64 + 16 + kNoticeBytes;  // and the groups' table, 16 bytes each
    static constexpr int kNAlign = PAIR ? 32 : 16;
    static constexpr int kWarpMma = 4, kWarpLoadP = 5, kWarpLoadQ = 6, kWarpLoadS = 7, kWarpScale = 8;
    static constexpr int kThreads = 32 * (kWarpScale + 1 + kQGroups);
    static_assert(kQBox % 8 == 0 && kStage % 1024 == 0, "1024-byte aligned operand tiles");
    static_assert(kTmemUse <= 512 && kOverlap >= 0 && kOverlap % 96 == 0, "TMEM budget");
    static_assert(!PAIR || BN == 256, "the pair form is built for 256 activation rows");
    static_assert(2 * 4 * 8 * 16 <= kStoreBytes, "notices of a split k");
};

struct Fp4Tile {
    int e;        // expert
    int p0;       // first weight row within the expert of this CTA
    int q0;       // first activation row (of all rows)
    int nq;       // activation rows of the tile
};

// A group in shared memory: its first tile, first activation row, rows and tiles
// of activations.
using Fp4Group = int4;

// Tile r of a group: the grouped order of its weight and activation tiles.
template <class Cfg>
__device__ __forceinline__ Fp4Tile fp4_tile_of(const Fp4Params &prm, int e, int begin, int count, int q_tiles, int r,
                                               int rank)
{
    Fp4Tile x;
    x.e = e;
    const int per_group = prm.group_p * q_tiles;
    const int grp = r / per_group;
    const int first = grp * prm.group_p;
    const int gsize = min(prm.p_tiles - first, prm.group_p);
    r -= grp * per_group;
    const int qi = r / gsize;
    x.p0 = ((first + r - qi * gsize) * Cfg::CL + rank) * 128;
    // equal tiles (of whole MMA columns): a short last one would load its weights
    // for little
    // (unsigned: rows and tiles together may pass 2^31)
    const int per = static_cast<int>((static_cast<uint32_t>(count) + q_tiles - 1) / q_tiles + Cfg::kNAlign - 1) &
                    ~(Cfg::kNAlign - 1);
    x.q0 = begin + qi * per;
    x.nq = min(count - qi * per, per);
    return x;
}

// Tile t: group by binary search over the first tiles.
template <class Cfg>
__device__ __forceinline__ Fp4Tile fp4_tile(const Fp4Params &prm, const Fp4Group *groups, int t, int rank)
{
    int begin = 0, count = prm.rows, r = t;
    int e = 0;
    int q_tiles = 0;
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
    return fp4_tile_of<Cfg>(prm, e, begin, count, q_tiles, r, rank);
}

// One warp, 32 groups from e0: this lane's group, with its first tile after `run`
// others; `run` moves past them.  (Groups that overlap against the rules could have
// more tiles than an int holds: those past kFp4MaxTiles are left out.)
template <class Params>
__device__ __forceinline__ Fp4Group fp4_groups32(const Params &prm, int e0, int &run)
{
    const int lane = threadIdx.x & 31, e = e0 + lane;
    Fp4Group g = make_int4(0, 0, 0, 0);
    if (e < prm.experts) {
        g.y = min(max(ld_relaxed_s32(prm.offsets + e), 0), prm.rows);
        g.z = min(max(ld_relaxed_s32(prm.offsets + e + 1), g.y), prm.rows) - g.y;
        g.w = (g.z + prm.qt - 1) / prm.qt;
    }
    int incl = g.w * prm.p_tiles;  // at most kFp4MaxTiles
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl = min(incl + o, kFp4MaxTiles);
    }
    const int before = __shfl_up_sync(0xffffffffu, incl, 1);
    g.x = min(run + (lane > 0 ? before : 0), kFp4MaxTiles);
    run = min(run + __shfl_sync(0xffffffffu, incl, 31), kFp4MaxTiles);
    return g;
}

// The weights of tile x that fill the ring first go to L2 while the kernel before
// this one ends.  (It may be the one that writes them: L2 then holds what it wrote,
// and the loads come after its end.)
__device__ __forceinline__ void fp4_prefetch(const Fp4Params &prm, const CUtensorMap *map, const Fp4Tile &x, int rank)
{
    if (elect_one()) {
        const int k0 = 2 * rank * prm.blocks_per_slice;
#pragma unroll 1
        for (int k = k0; k < min((prm.k_steps + 3) / 4, k0 + prm.prefetch); ++k)
            tma_prefetch_2d(map, k * 128, x.e * prm.N + x.p0);
    }
    __syncwarp();
}

__device__ __forceinline__ bool fp4_warp_wait(uint64_t *bar, uint32_t parity, const Watchdog &wd)
{
    const bool ok = wait_bounded(bar, parity, wd);
    return __all_sync(0xffffffffu, ok);
}

// Three barriers (their tests overlap when they are already complete).  PAIR: the third
// acquires at cluster scope, for what threads of the odd CTA wrote.
template <bool PAIR>
__device__ __forceinline__ bool fp4_warp_wait3(uint64_t *a, uint32_t pa, uint64_t *b, uint32_t pb, uint64_t *c,
                                               uint32_t pc, const Watchdog &wd)
{
    const bool ra = mbar_try_wait(a, pa), rb = mbar_try_wait(b, pb);
    const bool rc = PAIR ? mbar_try_wait_cluster(c, pc) : mbar_try_wait(c, pc);
    if (__all_sync(0xffffffffu, ra && rb && rc)) return true;
    const bool ok = wait_bounded(a, pa, wd) && wait_bounded(b, pb, wd) &&
                    (PAIR ? wait_bounded_cluster(c, pc, wd) : wait_bounded(c, pc, wd));
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool fp4_warp_wait_cluster(uint64_t *bar, uint32_t parity, const Watchdog &wd)
{
    const bool ok = wait_bounded_cluster(bar, parity, wd);
    return __all_sync(0xffffffffu, ok);
}

// Waits for the last phase of the ring slots in `issued` (their parities in `last`),
// all within one limit: at the end of a kernel that may have given up.
__device__ __forceinline__ void fp4_drain(uint64_t *bars, uint32_t issued, uint32_t last, uint64_t t0,
                                          unsigned long long limit_ns)
{
#pragma unroll 1
    for (int s = 0; issued >> s; ++s)
        if ((issued >> s) & 1u)
            while (!mbar_try_wait(&bars[s], (last >> s) & 1u) && globaltimer_ns() - t0 < limit_ns) {
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

// One value of C.
template <class Params>
__device__ __forceinline__ void fp4_store1(const Params &prm, float v, int64_t m, int n)
{
    if (n >= prm.N) return;
    const int64_t at = m * prm.N + n;
    if (prm.c_type == kOutF32)
        static_cast<float *>(prm.C)[at] = v;
    else if (prm.c_type == kOutBf16)
        static_cast<__nv_bfloat16 *>(prm.C)[at] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(prm.C)[at] = __float2half_rn(v);
}

// 32 accumulator columns (rows of C) of the warp's 32 lanes (columns of C).
// float32: thread = lane, its columns; a store is 128 contiguous bytes of a row.
// 16-bit: in fragment order (tmem_ld_16x256b_x2, lanes 0-15 then 16-31), turned by
// stmatrix so that a row's 32 columns are contiguous in the warp's 2 KB of
// shared memory (64-byte rows, 16-byte chunk c of row r at c ^ (r / 2 % 4)) and
// leave with wide stores.  (32 at a time, not 16: the way through shared memory is
// latency; the last tile of 256 columns takes 4700 cycles against 5700.)
template <bool F32>
__device__ __forceinline__ void fp4_load16_cols(uint32_t tacc, int c, uint32_t (&v)[16])
{
    if constexpr (F32) {
        tmem_ld_32x32b_x16(tacc + c, v);
    } else {
        tmem_ld_16x256b_x2(tacc + c, v);
        tmem_ld_16x256b_x2(tacc + (16u << 16) + c, v + 8);
    }
}

template <bool F32, class Params>
__device__ __forceinline__ void fp4_store32_cols(const Params &prm, const uint32_t (*v)[16], float alpha, int64_t m0,
                                                 int count, int n0, uint8_t *stage)
{
    const int lane = threadIdx.x & 31;
    if constexpr (F32) {
        if (n0 + lane < prm.N) {
            float *c = static_cast<float *>(prm.C) + m0 * prm.N + n0 + lane;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (j < count) *c = __uint_as_float(v[j / 16][j % 16]) * alpha;
                c += prm.N;
            }
        }
    } else {
        const bool bf16 = prm.c_type == kOutBf16;
        const uint32_t base = smem_u32(stage);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t pk[8];  // matrix (half h, rows + 8 s, columns 8 j): pk[4 h + 2 j + s]
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float lo = __uint_as_float(v[g][2 * i]) * alpha, hi = __uint_as_float(v[g][2 * i + 1]) * alpha;
                if (bf16) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
                    pk[i] = *reinterpret_cast<const uint32_t *>(&b);
                } else {
                    const __half2 b = __floats2half2_rn(lo, hi);
                    pk[i] = *reinterpret_cast<const uint32_t *>(&b);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 16 * g + 8 * j + (lane & 7), chunk = lane >> 3;
                stmatrix_x4_trans(base + r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4), pk[2 * j], pk[2 * j + 1],
                                  pk[4 + 2 * j], pk[4 + 2 * j + 1]);
            }
        }
        __syncwarp();
        uint16_t *c = static_cast<uint16_t *>(prm.C) + m0 * prm.N;
        if (prm.store_bytes == 16) {  // (N is a multiple of 8)
            uint4 q[4];
            const int chunk = lane & 3, n = n0 + 8 * chunk;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + (lane >> 2);
                q[i] = *reinterpret_cast<const uint4 *>(stage + r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + (lane >> 2);
                if (r < count && n < prm.N) *reinterpret_cast<uint4 *>(c + static_cast<int64_t>(r) * prm.N + n) = q[i];
            }
        } else if (prm.store_bytes == 4) {  // (N is even)
            uint32_t q[16];
            const int w = lane & 15, n = n0 + 2 * w;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = 2 * i + (lane >> 4);
                q[i] = *reinterpret_cast<const uint32_t *>(stage + r * 64 + (((w >> 2) ^ ((r >> 1) & 3)) << 4) +
                                                           4 * (w & 3));
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = 2 * i + (lane >> 4);
                if (r < count && n < prm.N)
                    *reinterpret_cast<uint32_t *>(c + static_cast<int64_t>(r) * prm.N + n) = q[i];
            }
        } else {
            const int n = n0 + lane;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 16) {
                uint16_t q[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = r0 + i;
                    q[i] = *reinterpret_cast<const uint16_t *>(stage + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) +
                                                               2 * (lane & 7));
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (r0 + i < count && n < prm.N) c[static_cast<int64_t>(r0 + i) * prm.N + n] = q[i];
            }
        }
        __syncwarp();  // read before the next columns overwrite it
    }
}

// A tile's accumulator to C; release() once its columns that the other
// accumulator shares (with no overlap: all) are in registers.
template <class Cfg, bool F32, class Release>
__device__ __forceinline__ void fp4_store_tile(const Fp4Params &prm, const Fp4Tile &x, uint32_t tacc, uint32_t ab,
                                               float alpha, int n0, uint8_t *stage, Release release)
{
    int c = 0, c_end = x.nq;
    if constexpr (Cfg::kOverlap > 0) {
        const int shared0 = ab ? 0 : Cfg::BN - Cfg::kOverlap;
#pragma unroll 1
        for (int s = shared0; s < shared0 + Cfg::kOverlap; s += 96) {
            uint32_t v[6][16];
#pragma unroll
            for (int i = 0; i < 6; ++i) fp4_load16_cols<F32>(tacc, s + 16 * i, v[i]);
#pragma unroll
            for (int i = 0; i < 6; i += 2) tmem_ld_wait_regs(v[i], v[i + 1]);
            if (s + 96 == shared0 + Cfg::kOverlap) release();
#pragma unroll
            for (int i = 0; i < 6; i += 2)
                if (s + 16 * i < x.nq)
                    fp4_store32_cols<F32>(prm, v + i, alpha, static_cast<int64_t>(x.q0) + s + 16 * i, x.nq - s - 16 * i,
                                          n0, stage);
        }
        c = ab ? Cfg::kOverlap : 0;
        c_end = min(x.nq, ab ? Cfg::BN : Cfg::BN - Cfg::kOverlap);
    }
#pragma unroll 1
    for (; c < c_end; c += 32) {
        uint32_t v[2][16];
        fp4_load16_cols<F32>(tacc, c, v[0]);
        fp4_load16_cols<F32>(tacc, c + 16, v[1]);
        tmem_ld_wait_regs(v[0], v[1]);
        if (Cfg::kOverlap == 0 && c + 32 >= c_end) release();
        fp4_store32_cols<F32>(prm, v, alpha, static_cast<int64_t>(x.q0) + c, c_end - c, n0, stage);
    }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    igemm_fp4_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                     const __grid_constant__ CUtensorMap mapQs, const __grid_constant__ CUtensorMap mapSP, const __grid_constant__ CUtensorMap mapSQ,
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
    uint64_t *sf_raw = empty + Cfg::kMaxStages;     // [scale stages] scale rows landed
    uint64_t *sf_full = sf_raw + Cfg::kMaxScaleStages;    // [scale stages] ... turned (scale warps; even CTA of a pair:
                                                          // and the odd CTA's, its relay's copy)
    uint64_t *sf_empty = sf_full + Cfg::kMaxScaleStages;  // [scale stages] consumed (MMA commit)
    uint64_t *acc_full = sf_empty + Cfg::kMaxScaleStages; // [2] accumulator complete (commit)
    uint64_t *acc_empty = acc_full + 2;             // [2] accumulator (its overlap) read by the epilogue warps
    uint64_t *mma_drain = acc_empty + 2;
    uint64_t *red_full = mma_drain + 1;             // [2][4] split k: the other CTAs' partials of this warp's part landed
    uint64_t *red_empty = red_full + 8;             // [2][4] ... and the other CTAs have read what this warp sent
                                                    // (their notices)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Cfg::kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *total_slot = reinterpret_cast<int *>(tmem_slot + 2);
    // 16 bytes for each notice of another CTA, never read: pairs [scale stages]; split k
    // [2][4][8 CTAs], in the epilogue's staging, which it does not use
    uint8_t *tail = smem + ((prm.off_bars + 8 * Cfg::kNumBars + 64 + 15) & ~15);
    uint8_t *notices = PAIR ? tail : smem + prm.off_store;
    Fp4Group *groups = reinterpret_cast<Fp4Group *>(tail + Cfg::kNoticeBytes);
    const uint8_t *fixed = smem + ((prm.off_bars + 8 * Cfg::kNumBars + 15) & ~15);  // 16 bytes that stay as they are

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int cs = PAIR ? 1 : prm.cs;
    const int csize = PAIR ? 2 : cs;
    const int rank = csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int pr = PAIR ? rank : 0;                 // half of the pair's tile
    const int cid = blockIdx.x / csize, ncl = gridDim.x / csize;
    const bool leader = !PAIR || rank == 0;

    if (warp == Cfg::kWarpLoadP) {
        if (lane < prm.code_stages) {
            mbar_init(&full[lane], 2);  // the two loading warps
            mbar_init(&empty[lane], 1);
        }
        if (lane < prm.scale_stages) {
            mbar_init(&sf_raw[lane], 1);
            mbar_init(&sf_empty[lane], 1);
            mbar_init(&sf_full[lane], 1 + Cfg::kQGroups);
        }
        if (lane < 2) {
            mbar_init(&acc_full[lane], 1);
            mbar_init(&acc_empty[lane], 4 * Cfg::CL);
        }
        if (cs > 1 && lane < 8) {
            mbar_init(&red_full[lane], 1);
            mbar_init(&red_empty[lane], 1);
        }
        if (lane == 0) {
            mbar_init(mma_drain, 1);
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
        // running tile counts of the groups (the offsets may come from the kernel before)
        if (prm.offsets) {
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
    if constexpr (!PAIR)
        if (warp == 3 && prm.prefetch > 0 && prm.offsets) {
            // the first tile by the offsets as they are now: if the kernel before is the
            // one that writes them, only the prefetch misses
            int run = 0;
            for (int e0 = 0; e0 < prm.experts && run <= cid; e0 += 32) {
                const Fp4Group g = fp4_groups32(prm, e0, run);
                const uint32_t mine = __ballot_sync(0xffffffffu, g.x <= cid && cid - g.x < g.w * prm.p_tiles);
                if (mine) {
                    const int from = 31 - __clz(static_cast<int>(mine));
                    const int r = cid - __shfl_sync(0xffffffffu, g.x, from), q_tiles = __shfl_sync(0xffffffffu, g.w, from);
                    fp4_prefetch(prm, &mapP, fp4_tile_of<Cfg>(prm, e0 + from, 0, 1, q_tiles, r, 0), rank);
                }
            }
        }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tiles = *total_slot;
    Fp4Tile first{};
    if (cid < tiles) first = fp4_tile<Cfg>(prm, groups, cid, pr);
    if constexpr (!PAIR)
        if (warp == 3 && prm.prefetch > 0 && !prm.offsets && cid < tiles) fp4_prefetch(prm, &mapP, first, rank);
    if (csize > 1) cluster_sync_all();  // the other CTAs' barriers are initialised
    // Up to here the kernel before this one in the stream may still run.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Watchdog wd{abort_flag, prm.status, prm.limit_ns};
    // this CTA's slice of k (split k: the cluster rank's), in blocks
    const int b0 = PAIR ? 0 : min(rank * prm.blocks_per_slice, prm.blocks);
    const int b1 = PAIR ? prm.blocks : min(b0 + prm.blocks_per_slice, prm.blocks);

    if (warp == Cfg::kWarpLoadP || warp == Cfg::kWarpLoadQ) {
        // ------------------------------------------------------------ codes
        const bool q_side = warp == Cfg::kWarpLoadQ;
        Fp4Ring cr(prm.code_stages);
        const bool stream = !PAIR && !q_side && prm.stream;
        const uint64_t evict_first = l2_policy_evict_first();
        uint32_t issued = 0, last = 0;
        bool ok = true;
        for (int t = cid; ok && t < tiles; t += ncl) {
            const Fp4Tile x = t == cid ? first : fp4_tile<Cfg>(prm, groups, t, pr);
            // activation rows that this CTA loads (pair: half of the tile's)
            const int mine = PAIR ? ((x.nq + Cfg::kNAlign - 1) & ~(Cfg::kNAlign - 1)) / 2 : x.nq;
            const bool small = q_side && Cfg::kQRows < Cfg::kQBox && mine <= 2 * Cfg::kQRows;
            const bool two = small && mine > Cfg::kQRows;
            const int y = q_side ? x.q0 + pr * mine : x.e * prm.N + x.p0;
            const uint32_t tx = static_cast<uint32_t>(
                !q_side ? Cfg::kBoxP : !small ? Cfg::kBoxQ : (two ? 2 : 1) * Cfg::kQRows * 128);
            const CUtensorMap *map = !q_side ? &mapP : small ? &mapQs : &mapQ;
            const uint32_t off = q_side ? Cfg::kBoxP : 0;
#pragma unroll 1
            for (int k = 2 * b0; k < 2 * b1; ++k) {
                if (!fp4_warp_wait(&empty[cr.slot], cr.phase ^ 1u, wd)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    uint8_t *to = codes + cr.slot * Cfg::kStage + off;
                    if constexpr (PAIR) {
                        // both CTAs' bytes count on the even CTA's barrier
                        if (leader) mbar_arrive_expect_tx(&full[cr.slot], 2 * tx);
                        const uint32_t bar = cluster_map(smem_u32(&full[cr.slot]), 0u);
                        tma_load_2d_pair(to, map, bar, k * 128, y);
                        if (two) tma_load_2d_pair(to + Cfg::kQRows * 128, map, bar, k * 128, y + Cfg::kQRows);
                    } else {
                        mbar_arrive_expect_tx(&full[cr.slot], tx);
                        // (a hint only where it says something: evict_normal for all loads
                        // took 1 x 4096 x 14336 from 7.3 to 8.4 us)
                        if (stream) tma_load_2d_hint(to, map, &full[cr.slot], k * 128, y, evict_first);
                        else tma_load_2d(to, map, &full[cr.slot], k * 128, y);
                        if (two) tma_load_2d(to + Cfg::kQRows * 128, map, &full[cr.slot], k * 128, y + Cfg::kQRows);
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
    } else if (warp == Cfg::kWarpLoadS) {
        // ------------------------------------------------------------ scale rows
        Fp4Ring sr(prm.scale_stages);
        uint32_t issued = 0, last = 0;
        bool ok = true;
        for (int t = cid; ok && t < tiles; t += ncl) {
            const Fp4Tile x = t == cid ? first : fp4_tile<Cfg>(prm, groups, t, pr);
            const int py = x.e * prm.N + x.p0;
            const int q_groups = (x.nq + 127) / 128;
            const uint32_t tx = static_cast<uint32_t>((128 + q_groups * Cfg::kQScaleRows) * 16 * Cfg::kH);
#pragma unroll 1
            for (int b = b0; b < b1; ++b) {
                if (!fp4_warp_wait(&sf_empty[sr.slot], sr.phase ^ 1u, wd)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    uint8_t *to = scales + sr.slot * Cfg::kScaleStage;
                    mbar_arrive_expect_tx(&sf_raw[sr.slot], tx);
                    tma_load_2d(to, &mapSP, &sf_raw[sr.slot], b * 16 * Cfg::kH, py);
#pragma unroll
                    for (int j = 0; j < Cfg::kQGroups; ++j)
                        if (j < q_groups)
                            tma_load_2d(to + Cfg::kGroupBytes * (1 + j), &mapSQ, &sf_raw[sr.slot], b * 16 * Cfg::kH,
                                        x.q0 + 128 * j);
                }
                __syncwarp();
                issued |= 1u << sr.slot;
                last = (last & ~(1u << sr.slot)) | (sr.phase << sr.slot);
                sr.next();
            }
        }
        const uint64_t t0 = globaltimer_ns();
        fp4_drain(sf_raw, issued, last, t0, prm.limit_ns);
        fp4_drain(sf_empty, issued, last, t0, prm.limit_ns);
    } else if (warp == Cfg::kWarpMma) {
        // ------------------------------------------------------------ MMA issuer
        if (leader) {
            Fp4Ring cr(prm.code_stages), fr(prm.scale_stages);
            const uint64_t desc0 = sdesc_kmajor_sw128(smem_u32(codes));
            const uint64_t sdesc0 = sdesc_rows16(smem_u32(scales));
            uint32_t nacc = 0, g = 0;
            const uint32_t slots = (1u << prm.scale_stages) - 1u;
            bool ok = true;
            for (int t = cid; ok && t < tiles; t += ncl, ++nacc) {
                const Fp4Tile x = t == cid ? first : fp4_tile<Cfg>(prm, groups, t, pr);
                const uint32_t nq = static_cast<uint32_t>((x.nq + Cfg::kNAlign - 1) & ~(Cfg::kNAlign - 1));
                const uint32_t idesc = idesc_fp4(128 * Cfg::CL, nq, NV);
                const uint32_t ab = nacc & 1u;
                const uint32_t d_tmem = tmem + ab * Cfg::kAcc1;
                if constexpr (Cfg::kOverlap > 0) {
                    // the tile before has left the columns that both accumulators use
                    ok = nacc == 0 || fp4_warp_wait(&acc_empty[ab ^ 1u], ((nacc - 1u) >> 1) & 1u, wd);
                } else {
                    ok = fp4_warp_wait(&acc_empty[ab], ((nacc >> 1) & 1u) ^ 1u, wd);
                }
                if (!ok) break;
                for (int b = b0; b < b1; ++b, ++g) {
                    const Fp4Ring c0 = cr;
                    cr.next();
                    if (!fp4_warp_wait3<PAIR>(&full[c0.slot], c0.phase, &full[cr.slot], cr.phase, &sf_full[fr.slot],
                                              fr.phase, wd)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t s0 = sdesc0 + static_cast<uint64_t>(fr.slot * (Cfg::kScaleStage >> 4));
                    const int steps = prm.k_steps - 8 * b;
                    // scale columns: mx the block's, alternating by block; nv a stage's each
                    const uint32_t sf = tmem + Cfg::kSf0 + (NV ? 0u : (g & 1u) * Cfg::kSfCols);
                    if (elect_one()) {
#pragma unroll
                        for (int h = 0; h < Cfg::kH; ++h)
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const uint64_t from = s0 + static_cast<uint64_t>((h * 2048 + w * 512) >> 4);
                                const uint32_t to = sf + h * Cfg::kSfCols;
                                tmem_cp_32x128b_x4<PAIR>(to + 4 * w, from);
#pragma unroll
                                for (int j = 0; j < Cfg::kQGroups; ++j)
                                    tmem_cp_32x128b_x4<PAIR>(
                                        to + 16 + Cfg::kQCols * w + 4 * j,
                                        from + static_cast<uint64_t>(((1 + j) * Cfg::kGroupBytes) >> 4));
                            }
                        // the scales' slot is free once they are in TMEM
                        if constexpr (PAIR)
                            mma_commit_pair_multicast(&sf_empty[fr.slot], 0x3);
                        else
                            mma_commit(&sf_empty[fr.slot]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int slot = h ? cr.slot : c0.slot;
                            const uint64_t p0 = desc0 + static_cast<uint64_t>(slot * (Cfg::kStage >> 4));
                            const uint64_t q0 = p0 + static_cast<uint64_t>(Cfg::kBoxP >> 4);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if (4 * h + q < steps) {
                                    // a word holds 64 k (nv) or 128 k (mx)
                                    const int word = NV ? q : 2 * h + q / 2;
                                    const uint32_t id = NV ? 0u : 2u * (q & 1);
                                    const uint32_t at = sf + (NV ? h * Cfg::kSfCols : 0);
                                    mma_fp4<NV, PAIR>(d_tmem, p0 + static_cast<uint64_t>(2 * q),
                                                      q0 + static_cast<uint64_t>(2 * q), idesc | (id << 4) | (id << 29),
                                                      at + 4 * word, at + 16 + Cfg::kQCols * word,
                                                      b > b0 || h > 0 || q > 0 ? 1u : 0u);
                                }
                            }
                            if constexpr (PAIR)
                                mma_commit_pair_multicast(&empty[slot], 0x3);
                            else
                                mma_commit(&empty[slot]);
                        }
                    }
                    __syncwarp();
                    cr.next();
                    fr.next();
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
            // gave up: the odd CTA's notices of the blocks ahead may be on their way here
            if (PAIR && !ok) {
                const uint32_t behind = (1u << fr.slot) - 1u;  // slots whose next phase is the other one
                fp4_drain(sf_full, slots, fr.phase ? slots & ~behind : behind, globaltimer_ns(), prm.limit_ns);
            }
            __syncwarp();
        } else {
            // relay of the odd CTA: each block whose scales are turned is announced to the
            // even CTA's MMA warp by copying 16 bytes of them there.  What the scale warps wrote
            // comes before this warp's wait, so before the copy (which reads it, through the
            // proxy of tcgen05.cp), so before the copy's completion, a release at cluster
            // scope that the MMA warp acquires.  An arrival with .release.cluster says the same
            // with a fence of its own, 1100 cycles and more: 8192^3 mx 240 us by one warp, 168
            // by two, 163 with copies (the three in turn); 512 x 8192 x 8192 26.7, 19.3, 17.3.
            const uint32_t peer = cluster_map(smem_u32(sf_full), 0u), notice = cluster_map(smem_u32(notices), 0u);
            Fp4Ring fr(prm.scale_stages);
            bool ok = true;
            for (int t = cid; ok && t < tiles; t += ncl) {
                for (int b = b0; b < b1; ++b) {
                    ok = fp4_warp_wait(&sf_full[fr.slot], fr.phase, wd);
                    if (!ok) break;
                    if (elect_one())
                        bulk_copy_to_cta(notice + 16u * static_cast<uint32_t>(fr.slot),
                                         scales + fr.slot * Cfg::kScaleStage, 16,
                                         peer + 8u * static_cast<uint32_t>(fr.slot));
                    __syncwarp();
                    fr.next();
                }
            }
        }
    } else if (warp >= Cfg::kWarpScale) {
        // ------------------------------------------------------------ scales
        // group 0: the tile's 128 weight rows; 1, 2: 128 activation rows each (a group
        // past the tile's rows has nothing new to turn: what it leaves there goes to
        // columns that no MMA of the tile reads)
        constexpr int H = Cfg::kH;
        const int group = warp - Cfg::kWarpScale;
        const int rows = group == 0 ? 128 : Cfg::kQScaleRows;  // of the box
        Fp4Ring fr(prm.scale_stages);
        bool ok = true;
        for (int t = cid; ok && t < tiles; t += ncl) {
            for (int b = b0; b < b1; ++b) {
                ok = fp4_warp_wait(&sf_raw[fr.slot], fr.phase, wd);
                if (!ok) break;
                uint4 *at = reinterpret_cast<uint4 *>(scales + fr.slot * Cfg::kScaleStage + group * Cfg::kGroupBytes);
                uint4 d[H][4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        d[h][j] = 32 * j + lane < rows ? at[(32 * j + lane) * H + h] : make_uint4(0, 0, 0, 0);
                __syncwarp();  // the warp's rows are read
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    // padding bytes past the last block of values count as zero scales
                    const int left = prm.k_blocks - 16 * (b * H + h);
                    if (left < 16) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            d[h][j] = make_uint4(fp4_keep(d[h][j].x, left), fp4_keep(d[h][j].y, left - 4),
                                                 fp4_keep(d[h][j].z, left - 8), fp4_keep(d[h][j].w, left - 12));
                    }
                    uint4 *to = at + 128 * h + lane;
                    to[0] = make_uint4(d[h][0].x, d[h][1].x, d[h][2].x, d[h][3].x);
                    to[32] = make_uint4(d[h][0].y, d[h][1].y, d[h][2].y, d[h][3].y);
                    to[64] = make_uint4(d[h][0].z, d[h][1].z, d[h][2].z, d[h][3].z);
                    to[96] = make_uint4(d[h][0].w, d[h][1].w, d[h][2].w, d[h][3].w);
                }
                fence_proxy_async_smem();  // read next by tcgen05.cp
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && leader && group == 0)
                        mbar_arrive_expect_tx(&sf_full[fr.slot], 16);  // the odd CTA's notice
                    else
                        mbar_arrive(&sf_full[fr.slot]);
                }
                fr.next();
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int quad = warp;
        const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        uint8_t *stage = smem + prm.off_store + quad * 2048;
        const uint32_t empty_leader = PAIR ? cluster_map(smem_u32(acc_empty), 0u) : 0u;
        uint32_t nacc = 0, armed = 0;  // armed: split k, tiles whose partials this warp expects
        bool ok = true;
        for (int t = cid; t < tiles; t += ncl, ++nacc) {
            const Fp4Tile x = t == cid ? first : fp4_tile<Cfg>(prm, groups, t, pr);
            const float alpha = prm.alpha ? prm.alpha[x.e] : 1.0f;
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
            ok = fp4_warp_wait(&acc_full[ab], (nacc >> 1) & 1u, wd);
            if (!ok) break;
            tc_fence_after();
            if (cs > 1) {
                // split k: every CTA sends its partial of columns r BN / cs .. to CTA r of the
                // cluster, which adds them in rank order (fixed, whatever arrives
                // first): four columns of 128 lanes are 2 KB at [rank][column / 4]
                const int per_log2 = __ffs(BN / cs) - 1, per = 1 << per_log2;
                const uint32_t rb = nacc % Cfg::kRedBufs, rph = (nacc / Cfg::kRedBufs) & 1u, bar = rb * 4 + quad;
                uint4 *buf = reinterpret_cast<uint4 *>(red) + rb * (BN * 32) + quad * 32 + lane;
                if (lane == 0) mbar_arrive_expect_tx(&red_full[bar], static_cast<uint32_t>((cs - 1) * per * 128));
                ++armed;
                ok = fp4_warp_wait_cluster(&red_empty[bar], rph ^ 1u, wd);
                if (!ok) break;
#pragma unroll 1
                for (int c0 = 0; c0 < BN; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(tacc + c0, v);
                    tmem_ld_wait_regs(v);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const int c = c0 + j, owner = c >> per_log2;
                        uint4 *to = buf + ((rank << per_log2) + (c & (per - 1))) / 4 * 128;
                        if (owner == rank)
                            *to = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                        else
                            st_async_v4(cluster_map(smem_u32(to), static_cast<uint32_t>(owner)), v + j,
                                        cluster_map(smem_u32(&red_full[bar]), static_cast<uint32_t>(owner)));
                    }
                }
                release();
                ok = fp4_warp_wait_cluster(&red_full[bar], rph, wd);
                if (!ok) break;
                const int c1 = min(per, x.nq - rank * per);
                for (int c = 0; c < c1; c += 4) {
                    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (int r = 0; r < cs; ++r) {
                        const uint4 v = buf[((r << per_log2) + c) / 4 * 128];
                        s[0] += __uint_as_float(v.x);
                        s[1] += __uint_as_float(v.y);
                        s[2] += __uint_as_float(v.z);
                        s[3] += __uint_as_float(v.w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (c + j < c1) fp4_store1(prm, s[j] * alpha, static_cast<int64_t>(x.q0) + rank * per + c + j, n);
                }
                __syncwarp();
                // read: the other CTAs may write again, where a later tile does.  Each is sent 16
                // bytes (no matter which): this warp's reads come before that copy, so before its
                // completion, a release at cluster scope, as with the pairs' relay.  (Arrivals
                // with .release.cluster wait for a fence: 64 x 28672 x 8192 mxfp4 25.1 us, 23.2
                // with copies.)
                if (t + static_cast<int64_t>(Cfg::kRedBufs) * ncl < tiles) {
                    if (lane == 0) mbar_arrive_expect_tx(&red_empty[bar], 16u * (cs - 1));
                    if (lane < cs && lane != rank)
                        bulk_copy_to_cta(cluster_map(smem_u32(notices + 16 * (8 * bar + rank)), lane), fixed, 16,
                                         cluster_map(smem_u32(&red_empty[bar]), lane));
                }
                continue;
            }
            const int n0 = x.p0 + quad * 32;
            if (prm.c_type == kOutF32)
                fp4_store_tile<Cfg, true>(prm, x, tacc, ab, alpha, n0, stage, release);
            else
                fp4_store_tile<Cfg, false>(prm, x, tacc, ab, alpha, n0, stage, release);
        }
        // gave up: another CTA's partials of this tile, and of the next with two buffers,
        // may be on their way here, and its notices of the tiles before
        if (cs > 1 && !ok) {
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t n = nacc > Cfg::kRedBufs ? nacc - Cfg::kRedBufs : 0u; n <= nacc; ++n)
                while (!mbar_try_wait(&red_empty[n % Cfg::kRedBufs * 4 + quad], (n / Cfg::kRedBufs) & 1u) &&
                       globaltimer_ns() - t0 < prm.limit_ns) {
                }
            for (uint32_t n = nacc; n < nacc + Cfg::kRedBufs; ++n) {
                uint64_t *bar = &red_full[n % Cfg::kRedBufs * 4 + quad];
                if (lane == 0 && n >= armed)
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>((cs - 1) * (BN / cs) * 128));
                while (!mbar_try_wait(bar, (n / Cfg::kRedBufs) & 1u) && globaltimer_ns() - t0 < prm.limit_ns) {
                }
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    // The next kernel may be set up on SMs that this one has left; it waits for the end
    // of this grid before it touches memory.  (Let in from the start, its blocks settle on
    // the SMs that happen to have room: 128 x 4096 x 4096 back to back 6.8 us against 6.5,
    // a mixture-of-experts layer of 8 tokens 52.5 against 49.)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (warp == Cfg::kWarpMma) {
        if (leader && lane == 0) fp4_drain(mma_drain, 1u, 0u, globaltimer_ns(), prm.limit_ns);
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
