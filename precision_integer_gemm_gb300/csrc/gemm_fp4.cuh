// Host side of the 4-bit floating-point GEMM: plan and launch of
// igemm_fp4_kernel for one format (the two formats are two translation units).
#pragma once
#include <atomic>
#include <cmath>
#include <mutex>
#include "launch.cuh"
#include "fp4.cuh"
#include "gemm_fp4_kernel.cuh"

namespace igemm {

// Shared memory of one launch: code stages, the ring of scales, the partials of a
// split k, the epilogue's staging, then barriers and the groups' table.
template <class Cfg>
struct Fp4Smem {
    int code_stages, scale_stages, off_scales, off_red, off_store, off_bars, total;
    Fp4Smem(int cs, int experts)
    {
        constexpr int kLimit = 227 * 1024 - 1024;  // less the alignment slack
        const int red = cs > 1 ? Cfg::kRedBytes : 0;
        const int tail = Cfg::kTailBytes + 16 * experts;
        const int left = kLimit - red - Cfg::kStoreBytes - tail;
        // (three blocks of scales at least: with two, nvfp4 8192^3 measured 176 us against
        // 166, although that leaves room for a sixth stage of codes)
        code_stages = std::min((left - 3 * Cfg::kScaleStage) / Cfg::kStage, static_cast<int>(Cfg::kMaxStages));
        scale_stages = std::min((left - code_stages * Cfg::kStage) / Cfg::kScaleStage,
                                static_cast<int>(Cfg::kMaxScaleStages));
        off_scales = code_stages * Cfg::kStage;
        off_red = off_scales + scale_stages * Cfg::kScaleStage;
        off_store = off_red + red;
        off_bars = off_store + Cfg::kStoreBytes;
        total = off_bars + tail + 1024;
    }
};

// Clusters of `csize` CTAs of igemm_fp4_kernel<Cfg> that can be resident at once, 0 if
// none fits (asked once per device and size); sets the kernel's shared-memory limit.
template <class Cfg>
int fp4_clusters(int csize)
{
    static std::mutex mu;
    // one more than the clusters (a small call asks several times: no lock once known)
    static std::atomic<int> cache[64][4] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    const int slot = csize == 1 ? 0 : csize == 2 ? 1 : csize == 4 ? 2 : 3;
    if (const int known = cache[dev][slot].load(std::memory_order_acquire)) return known - 1;
    std::lock_guard<std::mutex> lock(mu);
    if (!cache[dev][slot]) {
        auto kernel = igemm_fp4_kernel<Cfg>;
        int n = sm_count();
        cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (rc == cudaSuccess && csize > 1) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = csize;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(csize * sm_count(), 1, 1);
            cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
            cfg.dynamicSmemBytes = 227 * 1024;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            rc = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        }
        if (rc != cudaSuccess) {
            cudaGetLastError();  // (the launch of another kernel is not to report it)
            return 0;
        }
        cache[dev][slot].store(std::max(n, 0) + 1, std::memory_order_release);
    }
    return cache[dev][slot] - 1;
}

template <class Cfg>
int launch_fp4_cfg(const Fp4Call &c, const Fp4Plan &plan, cudaStream_t stream)
{
    const int csize = Cfg::PAIR ? 2 : plan.cs;
    const int clusters = fp4_clusters<Cfg>(csize);
    if (clusters < 1) return kCudaError;
    const int code_bytes = fp4_code_bytes(c.K), pitch = fp4_scale_pitch(c.K, Cfg::NV);
    const uint64_t p_rows = uint64_t(c.experts) * c.N;
    CUtensorMap mapP, mapQ, mapQs, mapSP, mapSQ;
    constexpr CUtensorMapDataType kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (make_map(&mapP, kU8, c.B, p_rows, code_bytes, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) != kOk ||
        make_map(&mapQ, kU8, c.A, c.rows, code_bytes, Cfg::kQBox, 128, CU_TENSOR_MAP_SWIZZLE_128B) != kOk ||
        make_map(&mapSP, kU8, c.SFB, p_rows, pitch, 128, 16 * Cfg::kH, CU_TENSOR_MAP_SWIZZLE_NONE) != kOk ||
        make_map(&mapSQ, kU8, c.SFA, c.rows, pitch, Cfg::kQScaleRows, 16 * Cfg::kH,
                 CU_TENSOR_MAP_SWIZZLE_NONE) != kOk)
        return kCudaError;
    if constexpr (Cfg::kQRows == Cfg::kQBox)
        mapQs = mapQ;
    else if (make_map(&mapQs, kU8, c.A, c.rows, code_bytes, Cfg::kQRows, 128, CU_TENSOR_MAP_SWIZZLE_128B) != kOk)
        return kCudaError;
    const Fp4Smem<Cfg> lay(Cfg::PAIR ? 1 : csize, c.offsets ? c.experts : 0);
    Fp4Params prm{};
    prm.C = c.C;
    prm.c_type = c.c_type;
    prm.alpha = c.alpha;
    prm.offsets = c.offsets;
    prm.rows = c.rows;
    prm.N = c.N;
    prm.experts = c.experts;
    prm.k_steps = (c.K + 63) / 64;
    prm.k_blocks = (c.K + (Cfg::NV ? 15 : 31)) / (Cfg::NV ? 16 : 32);
    prm.blocks = (c.K + 511) / 512;
    prm.qt = plan.qt;
    prm.p_tiles = (c.N + 128 * Cfg::CL - 1) / (128 * Cfg::CL);
    prm.group_p = plan.group_p;
    prm.cs = plan.cs;
    prm.blocks_per_slice = (prm.blocks + plan.cs - 1) / plan.cs;
    // weights from 24 MB on leave L2 first, before what other kernels left there (us
    // without and with: 32 rows over 64 experts of 4096 x 4096 39.2 to 36.1, 16 x 28672 x
    // 8192 nvfp4 24.0 to 21.7, mxfp4 23.0 to 20.2; weights that L2 holds from call to call,
    // 64 x 14336 x 4096 7.6 to 7.9)
    const double weights = plan.groups * c.N * code_bytes;
    prm.stream = !Cfg::PAIR && weights >= 24.0 * (1 << 20);
    // weights of 32 MB and more, whose first ring is a small part of what a CTA reads (us
    // without and with: 16 x 28672 x 8192 mxfp4 22.5 to 20.2, nvfp4 21.8 to 21.7, 32 rows
    // over 64 experts of 4096 x 4096 37.9 to 36.1; with this hint and the one above for
    // smaller weights, 16 x 4096 x 4096 5.7 to 6.2, 1 x 4096 x 14336 8.1 to 8.8)
    prm.prefetch = !Cfg::PAIR && weights >= 32.0 * (1 << 20)
                       ? std::min(lay.code_stages, 2 * prm.blocks_per_slice)
                       : 0;
    prm.code_stages = lay.code_stages;
    prm.scale_stages = lay.scale_stages;
    prm.off_scales = lay.off_scales;
    prm.off_red = lay.off_red;
    prm.off_store = lay.off_store;
    prm.off_bars = lay.off_bars;
    const uintptr_t rows_at = reinterpret_cast<uintptr_t>(c.C) | (static_cast<uintptr_t>(c.N) * 2);
    prm.store_bytes = rows_at % 16 == 0 ? 16 : rows_at % 4 == 0 ? 4 : 2;
    prm.status = device_status_word();
    prm.limit_ns = watchdog_limit_ns();
    if (!prm.status) return kCudaError;
    // every slice of k holds at least one block
    if (plan.cs > 1 && prm.blocks_per_slice * (plan.cs - 1) >= prm.blocks) return kUnsupportedShape;
    const int64_t q_tiles = (int64_t(c.rows) + plan.qt - 1) / plan.qt + (c.offsets ? std::min(c.rows, c.experts) - 1 : 0);
    const int64_t tiles = q_tiles * prm.p_tiles;  // grouped: at most
    const GemmEvents ev = take_gemm_events();
    if (ev.start && cudaEventRecord(ev.start, stream) != cudaSuccess) return kCudaError;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int na = 0;
    // set up while the kernel before ends (with the timing events armed, the event
    // between the two keeps them apart)
    if (!ev.start) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    if (csize > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = csize;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(csize * std::min<int64_t>(tiles, clusters)), 1, 1);
    cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
    cfg.dynamicSmemBytes = lay.total;
    cfg.stream = stream;
    cfg.attrs = na ? attr : nullptr;
    cfg.numAttrs = na;
    if (cudaLaunchKernelEx(&cfg, igemm_fp4_kernel<Cfg>, mapP, mapQ, mapQs, mapSP, mapSQ, prm) != cudaSuccess)
        return kCudaError;
    note_launch();
    if (ev.stop && cudaEventRecord(ev.stop, stream) != cudaSuccess) return kCudaError;
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

template <bool NV>
int fp4_max_clusters(int bn, bool pair, int csize)
{
    if (pair) return fp4_clusters<Fp4Cfg<NV, 256, true>>(2);
    switch (bn) {
    case 16: return fp4_clusters<Fp4Cfg<NV, 16, false>>(csize);
    case 32: return fp4_clusters<Fp4Cfg<NV, 32, false>>(csize);
    case 64: return fp4_clusters<Fp4Cfg<NV, 64, false>>(csize);
    default: return fp4_clusters<Fp4Cfg<NV, 128, false>>(csize);
    }
}

template <bool NV>
int launch_fp4_format(const Fp4Call &c, cudaStream_t stream)
{
    Fp4Plan plan;
    if (!fp4_plan(c, fp4_max_clusters<NV>, &plan)) return kCudaError;
    if (plan.pair) return launch_fp4_cfg<Fp4Cfg<NV, 256, true>>(c, plan, stream);
    switch (plan.bn) {
    case 16: return launch_fp4_cfg<Fp4Cfg<NV, 16, false>>(c, plan, stream);
    case 32: return launch_fp4_cfg<Fp4Cfg<NV, 32, false>>(c, plan, stream);
    case 64: return launch_fp4_cfg<Fp4Cfg<NV, 64, false>>(c, plan, stream);
    default: return launch_fp4_cfg<Fp4Cfg<NV, 128, false>>(c, plan, stream);
    }
}

}  // namespace igemm
