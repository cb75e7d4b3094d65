// The experts' products with bf16 rows.
#include "mx_gemm_host.cuh"

namespace qgemv {
int launch_mx_gemm_bf16(int mode, const MxArgs& a, cudaStream_t s) { return launch_mx_gemm_t<__nv_bfloat16>(mode, a, s); }
}  // namespace qgemv
