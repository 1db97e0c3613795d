// Host side of the block-scaled fp8 GEMM: launch of igemm_bsfp8_kernel.
#include <atomic>
#include <mutex>
#include "launch.cuh"
#include "bsfp8.cuh"
#include "gemm_bsfp8_kernel.cuh"

namespace igemm {

// Shared memory of one launch: code stages, the ring of scales, the partials of a
// split k, the epilogue's staging, then barriers and the groups' table.
template <class Cfg>
struct Bsfp8Smem {
    int stages, off_scales, off_red, off_store, off_bars, total;
    Bsfp8Smem(int cs, int experts)
    {
        constexpr int kLimit = 227 * 1024 - 1024;  // less the alignment slack
        const int red = cs > 1 ? Cfg::kRedBytes : 0;
        const int tail = Cfg::kTailBytes + 16 * experts;
        const int left = kLimit - red - Cfg::kStoreBytes - Cfg::SS * Cfg::kScaleStage - tail;
        stages = std::min(left / Cfg::kStage, static_cast<int>(Cfg::kMaxStages));
        off_scales = stages * Cfg::kStage;
        off_red = off_scales + Cfg::SS * Cfg::kScaleStage;
        off_store = off_red + red;
        off_bars = off_store + Cfg::kStoreBytes;
        total = off_bars + tail + 1024;
    }
};

// Clusters of `csize` CTAs of igemm_bsfp8_kernel<Cfg> that can be resident at once, 0
// if none fits, below 0 where the runtime does not say; sets the kernel's shared-memory limit.
template <class Cfg>
int bsfp8_ask_clusters(int csize)
{
    auto kernel = igemm_bsfp8_kernel<Cfg>;
    int n = sm_count();
    cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (Cfg::PAIR && rc == cudaSuccess) {
        // the warps' shares of registers are dealt out of 168 a thread
        cudaFuncAttributes attr;
        rc = cudaFuncGetAttributes(&attr, kernel);
        if (rc == cudaSuccess && attr.numRegs != 168) return 0;
    }
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
        return -1;
    }
    return std::max(n, 0);
}

// ... asked once per device and size.
template <class Cfg>
int bsfp8_clusters(int csize)
{
    static std::mutex mu;
    static std::atomic<int> known[64][3] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    return bsfp8_ask_once(known[dev][csize == 1 ? 0 : csize == 2 ? 1 : 2], mu, [&] { return bsfp8_ask_clusters<Cfg>(csize); });
}

template <class Cfg>
static int launch_bsfp8_cfg(const Bsfp8Call &c, const Bsfp8Plan &plan, cudaStream_t stream)
{
    const int csize = Cfg::PAIR ? 2 : plan.cs;
    const int clusters = bsfp8_clusters<Cfg>(csize);
    if (clusters < 1) return kCudaError;
    const uint64_t p_rows = uint64_t(c.experts) * c.N, pitch = bsfp8_code_bytes(c.K);
    const int n_blocks = (c.N - 1) / 128 + 1, sf_bytes = bsfp8_scale_pitch(c.K) * 4;
    CUtensorMap mapP, mapQ, mapQs, mapSP, mapSQ;
    constexpr CUtensorMapDataType kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    // (K columns: bytes past them are zeros whatever the rows' padding holds)
    if (make_map(&mapP, kU8, c.B, p_rows, c.K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B, pitch) != kOk ||
        make_map(&mapQ, kU8, c.A, c.rows, c.K, Cfg::kQBox, 128, CU_TENSOR_MAP_SWIZZLE_128B, pitch) != kOk ||
        make_map(&mapSP, kU8, c.SFB, uint64_t(c.experts) * n_blocks, sf_bytes, Cfg::CL, 16,
                 CU_TENSOR_MAP_SWIZZLE_NONE) != kOk ||
        make_map(&mapSQ, kU8, c.SFA, c.rows, sf_bytes, Cfg::BN, 16, CU_TENSOR_MAP_SWIZZLE_NONE) != kOk)
        return kCudaError;
    if constexpr (Cfg::kQRows == Cfg::kQBox)
        mapQs = mapQ;
    else if (make_map(&mapQs, kU8, c.A, c.rows, c.K, Cfg::kQRows, 128, CU_TENSOR_MAP_SWIZZLE_128B, pitch) != kOk)
        return kCudaError;
    const Bsfp8Smem<Cfg> lay(Cfg::PAIR ? 1 : csize, c.offsets ? c.experts : 0);
    if (lay.stages < 2) return kUnsupportedShape;
    Bsfp8Params prm{};
    prm.C = c.C;
    prm.c_type = c.c_type;
    prm.offsets = c.offsets;
    prm.rows = c.rows;
    prm.N = c.N;
    prm.experts = c.experts;
    prm.blocks = (c.K + 127) / 128;
    prm.qt = Cfg::BN;
    prm.p_tiles = (c.N - 1) / (128 * Cfg::CL) + 1;
    prm.n_blocks = n_blocks;
    prm.group_p = plan.group_p;
    prm.cs = plan.cs;
    prm.slice = ((prm.blocks + 3) / 4 + plan.cs - 1) / plan.cs * 4;
    // every slice of k holds at least one block
    if (plan.cs > 1 && prm.slice * (plan.cs - 1) >= prm.blocks) return kUnsupportedShape;
    prm.stream = plan.stream;
    prm.format = c.format;
    const uintptr_t rows_at = reinterpret_cast<uintptr_t>(c.C) | (static_cast<uintptr_t>(c.N) * (c.c_type == kOutF32 ? 4 : 2));
    prm.store_bytes = rows_at % 16 == 0 ? 16 : rows_at % 4 == 0 ? 4 : 2;
    prm.wide = rows_at % 32 == 0;
    prm.stages = lay.stages;
    prm.off_scales = lay.off_scales;
    prm.off_red = lay.off_red;
    prm.off_store = lay.off_store;
    prm.off_bars = lay.off_bars;
    prm.status = device_status_word();
    prm.limit_ns = watchdog_limit_ns();
    prm.limit_ns32 = static_cast<uint32_t>(std::min<unsigned long long>(prm.limit_ns, 4000000000ull));
    if (!prm.status) return kCudaError;
    const int64_t q_tiles = (int64_t(c.rows) + Cfg::BN - 1) / Cfg::BN + (c.offsets ? std::min(c.rows, c.experts) - 1 : 0);
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
    if (cudaLaunchKernelEx(&cfg, igemm_bsfp8_kernel<Cfg>, mapP, mapQ, mapQs, mapSP, mapSQ, prm) != cudaSuccess)
        return kCudaError;
    note_launch();
    if (ev.stop && cudaEventRecord(ev.stop, stream) != cudaSuccess) return kCudaError;
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

static int bsfp8_max_clusters(int bn, bool pair, int csize)
{
    if (pair) return bsfp8_clusters<Bsfp8Cfg<256, true>>(2);
    switch (bn) {
    case 16: return bsfp8_clusters<Bsfp8Cfg<16, false>>(csize);
    case 32: return bsfp8_clusters<Bsfp8Cfg<32, false>>(csize);
    case 64: return bsfp8_clusters<Bsfp8Cfg<64, false>>(csize);
    default: return bsfp8_clusters<Bsfp8Cfg<128, false>>(csize);
    }
}

int launch_bsfp8(const Bsfp8Call &c, cudaStream_t stream)
{
    Bsfp8Plan plan;
    if (!bsfp8_plan(c, bsfp8_max_clusters, &plan)) return kCudaError;
    if (plan.pair) return launch_bsfp8_cfg<Bsfp8Cfg<256, true>>(c, plan, stream);
    switch (plan.bn) {
    case 16: return launch_bsfp8_cfg<Bsfp8Cfg<16, false>>(c, plan, stream);
    case 32: return launch_bsfp8_cfg<Bsfp8Cfg<32, false>>(c, plan, stream);
    case 64: return launch_bsfp8_cfg<Bsfp8Cfg<64, false>>(c, plan, stream);
    default: return launch_bsfp8_cfg<Bsfp8Cfg<128, false>>(c, plan, stream);
    }
}

}  // namespace igemm
