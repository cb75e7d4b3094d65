// The experts' products with fp32 rows.
#include "mx_gemm_host.cuh"

namespace qgemv {
int launch_mx_gemm_f32(int mode, const MxArgs& a, cudaStream_t s) { return launch_mx_gemm_t<float>(mode, a, s); }
}  // namespace qgemv
