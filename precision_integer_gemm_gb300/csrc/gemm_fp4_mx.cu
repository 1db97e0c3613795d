// The mx (ue8m0 scales per 32 k) instances of the 4-bit floating-point GEMM.
#include "gemm_fp4.cuh"

namespace igemm {

int launch_fp4_mx(const Fp4Call &c, cudaStream_t stream) { return launch_fp4_format<false>(c, stream); }

}  // namespace igemm
