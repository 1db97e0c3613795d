// C-ABI entry points of the block-scaled fp8 operators (declared in include/igemm.h):
// argument validation and dispatch.
#include <cstdint>
#include "launch.cuh"
#include "bsfp8.cuh"
#include "igemm.h"

using namespace igemm;

static bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
static bool known_type(int type) { return type >= IGEMM_F32 && type <= IGEMM_F16; }
static bool known_format(int format) { return format == IGEMM_E4M3 || format == IGEMM_E5M2; }
static int type_bytes(int type) { return type == IGEMM_F32 ? 4 : 2; }

extern "C" int pack_bsfp8(const void *x, int x_type, int64_t ld, int transposed, const int32_t *index, int x_rows,
                          int tile_rows, int format, uint8_t *codes, float *scales, int rows, int K,
                          cudaStream_t stream)
{
    if (rows < 0 || K < 0 || x_rows < 0 || ld < 0 || !known_type(x_type) || !known_format(format))
        return kInvalidArgument;
    if (tile_rows != 1 && tile_rows != 128) return kUnsupportedShape;
    if (rows == 0 || K == 0) return kOk;
    if (!codes || !scales || (!x && x_rows > 0)) return kInvalidArgument;
    if (index && (transposed || tile_rows != 1)) return kUnsupportedShape;
    if (!index && x_rows < rows) return kInvalidArgument;
    if (ld < (transposed ? x_rows : K)) return kInvalidArgument;
    if (K > IGEMM_BSFP8_MAX_K) return kOverflowBound;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(x, type_bytes(x_type)) || !aligned(index, 4))
        return kMisaligned;
    return launch_bsfp8_pack({format, x, x_type, ld, transposed != 0, index, x_rows, tile_rows, codes, scales, rows, K},
                             stream);
}

static int gemm_checked(const Bsfp8Call &c, bool grouped, cudaStream_t stream)
{
    if (c.rows < 0 || c.N < 0 || c.K < 0 || c.experts < 0 || !known_type(c.c_type) || !known_format(c.format))
        return kInvalidArgument;
    if (c.rows == 0 || c.N == 0 || c.experts == 0) return kOk;
    if (!c.C || (grouped && !c.offsets)) return kInvalidArgument;
    if (c.experts > kBsfp8MaxExperts || int64_t(c.experts) * c.N > 0x7FFFFFFF - 512 || c.rows > 0x7FFFFFFF - 512)
        return kUnsupportedShape;
    // tile numbers stay within int (tiles of 16 rows by 128 columns)
    if ((int64_t(c.rows) / 16 + c.experts) * ((int64_t(c.N) + 127) / 128) > kBsfp8MaxTiles) return kUnsupportedShape;
    if (c.K > IGEMM_BSFP8_MAX_K) return kOverflowBound;
    if (!aligned(c.C, type_bytes(c.c_type)) || !aligned(c.offsets, 4)) return kMisaligned;
    if (c.K == 0) {
        if (grouped) return kUnsupportedShape;
        return cudaMemsetAsync(c.C, 0, size_t(c.rows) * size_t(c.N) * type_bytes(c.c_type), stream) == cudaSuccess
                   ? kOk
                   : kCudaError;
    }
    if (!c.A || !c.B || !c.SFA || !c.SFB) return kInvalidArgument;
    if (!aligned(c.A, 16) || !aligned(c.B, 16) || !aligned(c.SFA, 16) || !aligned(c.SFB, 16)) return kMisaligned;
    return launch_bsfp8(c, stream);
}

extern "C" int igemm_bsfp8(const uint8_t *A, const uint8_t *B, const float *SFA, const float *SFB, void *C, int c_type,
                           int format, int M, int N, int K, cudaStream_t stream)
{
    return gemm_checked({format, A, B, SFA, SFB, nullptr, C, c_type, M, 1, N, K}, false, stream);
}

extern "C" int igemm_bsfp8_grouped(const uint8_t *A, const uint8_t *B, const float *SFA, const float *SFB,
                                   const int32_t *offsets, void *C, int c_type, int format, int rows, int E, int N, int K,
                                   cudaStream_t stream)
{
    return gemm_checked({format, A, B, SFA, SFB, offsets, C, c_type, rows, E, N, K}, true, stream);
}
