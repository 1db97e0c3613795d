// The nv (ue4m3 scales per 16 k) instances of the 4-bit floating-point GEMM.
#include "gemm_fp4.cuh"

namespace igemm {

int launch_fp4_nv(const Fp4Call &c, cudaStream_t stream) { return launch_fp4_format<true>(c, stream); }

}  // namespace igemm
