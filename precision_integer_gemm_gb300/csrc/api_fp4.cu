// C-ABI entry points of the 4-bit floating-point mixture-of-experts operators
// (declared in include/igemm.h): argument validation and dispatch.
#include <cstdint>
#include "launch.cuh"
#include "fp4.cuh"
#include "gemm_fp4_kernel.cuh"
#include "moe.cuh"
#include "igemm.h"

using namespace igemm;

static bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
static bool known_type(int type) { return type >= IGEMM_F32 && type <= IGEMM_F16; }
static int type_bytes(int type) { return type == IGEMM_F32 ? 4 : 2; }

static int pack_checked(Fp4PackCall c, cudaStream_t stream)
{
    if (c.rows < 0 || c.K < 0 || c.x_rows < 0 || c.ld < 0 || !known_type(c.x_type)) return kInvalidArgument;
    if (c.rows == 0 || c.K == 0) return kOk;
    if (!c.codes || !c.scales || (!c.x && c.x_rows > 0)) return kInvalidArgument;
    if (c.index && c.transposed) return kUnsupportedShape;
    if (!c.index && c.x_rows < c.rows) return kInvalidArgument;
    if (c.ld < (c.transposed ? c.x_rows : c.K)) return kInvalidArgument;
    if (c.K > IGEMM_FP4_MAX_K) return kOverflowBound;
    if (!aligned(c.codes, 16) || !aligned(c.scales, 16) || !aligned(c.x, type_bytes(c.x_type)) ||
        !aligned(c.index, 4) || !aligned(c.tensor_scale, 4))
        return kMisaligned;
    return launch_fp4_pack(c, stream);
}

extern "C" int pack_mxfp4(const void *x, int x_type, int64_t ld, int transposed, const int32_t *index, int x_rows,
                          uint8_t *codes, uint8_t *scales, int rows, int K, cudaStream_t stream)
{
    return pack_checked({false, x, x_type, ld, transposed != 0, index, x_rows, nullptr, codes, scales, rows, K},
                        stream);
}

extern "C" int pack_nvfp4(const void *x, int x_type, int64_t ld, int transposed, const int32_t *index, int x_rows,
                          const float *tensor_scale, uint8_t *codes, uint8_t *scales, int rows, int K,
                          cudaStream_t stream)
{
    return pack_checked({true, x, x_type, ld, transposed != 0, index, x_rows, tensor_scale, codes, scales, rows, K},
                        stream);
}

static int gemm_checked(const Fp4Call &c, bool grouped, cudaStream_t stream)
{
    if (c.rows < 0 || c.N < 0 || c.K < 0 || c.experts < 0 || !known_type(c.c_type)) return kInvalidArgument;
    if (c.rows == 0 || c.N == 0 || c.experts == 0) return kOk;
    if (!c.C || (grouped && !c.offsets)) return kInvalidArgument;
    if (c.experts > kFp4MaxExperts || int64_t(c.experts) * c.N > 0x7FFFFFFF - 512 || c.rows > 0x7FFFFFFF - 512)
        return kUnsupportedShape;
    // tile numbers stay within int (tiles of 16 rows by 128 columns)
    if ((int64_t(c.rows) / 16 + c.experts) * ((int64_t(c.N) + 127) / 128) > kFp4MaxTiles) return kUnsupportedShape;
    if (c.K > IGEMM_FP4_MAX_K) return kOverflowBound;
    if (!aligned(c.C, type_bytes(c.c_type)) || !aligned(c.alpha, 4) || !aligned(c.offsets, 4)) return kMisaligned;
    if (c.K == 0) {
        if (grouped) return kUnsupportedShape;
        return cudaMemsetAsync(c.C, 0, size_t(c.rows) * size_t(c.N) * type_bytes(c.c_type), stream) == cudaSuccess
                   ? kOk
                   : kCudaError;
    }
    if (!c.A || !c.B || !c.SFA || !c.SFB) return kInvalidArgument;
    if (!aligned(c.A, 16) || !aligned(c.B, 16) || !aligned(c.SFA, 16) || !aligned(c.SFB, 16)) return kMisaligned;
    return c.nv ? launch_fp4_nv(c, stream) : launch_fp4_mx(c, stream);
}

extern "C" int igemm_mxfp4(const uint8_t *A, const uint8_t *B, const uint8_t *SFA, const uint8_t *SFB, void *C,
                           int c_type, int M, int N, int K, cudaStream_t stream)
{
    return gemm_checked({false, A, B, SFA, SFB, nullptr, nullptr, C, c_type, M, 1, N, K}, false, stream);
}

extern "C" int igemm_nvfp4(const uint8_t *A, const uint8_t *B, const uint8_t *SFA, const uint8_t *SFB,
                           const float *alpha, void *C, int c_type, int M, int N, int K, cudaStream_t stream)
{
    return gemm_checked({true, A, B, SFA, SFB, nullptr, alpha, C, c_type, M, 1, N, K}, false, stream);
}

extern "C" int igemm_mxfp4_grouped(const uint8_t *A, const uint8_t *B, const uint8_t *SFA, const uint8_t *SFB,
                                   const int32_t *offsets, void *C, int c_type, int rows, int E, int N, int K,
                                   cudaStream_t stream)
{
    return gemm_checked({false, A, B, SFA, SFB, offsets, nullptr, C, c_type, rows, E, N, K}, true, stream);
}

extern "C" int igemm_nvfp4_grouped(const uint8_t *A, const uint8_t *B, const uint8_t *SFA, const uint8_t *SFB,
                                   const int32_t *offsets, const float *alpha, void *C, int c_type, int rows, int E,
                                   int N, int K, cudaStream_t stream)
{
    return gemm_checked({true, A, B, SFA, SFB, offsets, alpha, C, c_type, rows, E, N, K}, true, stream);
}

extern "C" int igemm_moe_route(const void *logits, int logits_type, int32_t *experts, float *weights,
                               int32_t *offsets, int32_t *tokens, int32_t *slots, int T, int E, int k, int normalize,
                               cudaStream_t stream)
{
    if (T < 0 || E < 0 || k < 0 || !known_type(logits_type)) return kInvalidArgument;
    if (!offsets) return kInvalidArgument;
    if (!aligned(offsets, 4)) return kMisaligned;
    if (E > kFp4MaxExperts || k > 32 || k > E || int64_t(T) * k > 0x7FFFFFFF) return kUnsupportedShape;
    if (T == 0 || k == 0)
        return cudaMemsetAsync(offsets, 0, size_t(E + 1) * 4, stream) == cudaSuccess ? kOk : kCudaError;
    if (!logits || !experts || !weights || !tokens || !slots) return kInvalidArgument;
    if (!aligned(logits, type_bytes(logits_type)) || !aligned(experts, 4) || !aligned(weights, 4) ||
        !aligned(tokens, 4) || !aligned(slots, 4))
        return kMisaligned;
    return launch_moe_route({logits, logits_type, experts, weights, offsets, tokens, slots, T, E, k, normalize != 0},
                            stream);
}

extern "C" int igemm_moe_combine(const void *Y, const int32_t *slots, const float *weights, void *out, int type, int T,
                                 int k, int N, cudaStream_t stream)
{
    if (T < 0 || k < 0 || N < 0 || !known_type(type)) return kInvalidArgument;
    if (T == 0 || N == 0) return kOk;
    if (!out) return kInvalidArgument;
    if (k > 32 || int64_t(T) * k > 0x7FFFFFFF) return kUnsupportedShape;
    if (!aligned(out, type_bytes(type))) return kMisaligned;
    if (k == 0)
        return cudaMemsetAsync(out, 0, size_t(T) * size_t(N) * type_bytes(type), stream) == cudaSuccess ? kOk
                                                                                                        : kCudaError;
    if (!Y || !slots || !weights) return kInvalidArgument;
    if (!aligned(Y, type_bytes(type)) || !aligned(slots, 4) || !aligned(weights, 4)) return kMisaligned;
    return launch_moe_combine({Y, type, slots, weights, out, T, k, N}, stream);
}
