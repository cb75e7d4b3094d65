// The experts' products with fp16 rows.
#include "mx_gemm_host.cuh"

namespace qgemv {
int launch_mx_gemm_f16(int mode, const MxArgs& a, cudaStream_t s) { return launch_mx_gemm_t<__half>(mode, a, s); }
}  // namespace qgemv
