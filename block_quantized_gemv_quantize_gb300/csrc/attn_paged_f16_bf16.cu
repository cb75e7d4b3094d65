// attn_paged over f16 pages for bf16 rows.
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_f16_bf16(const AttnArgs& a, cudaStream_t s) { return launch_attn_rows<QGEMV_KV_F16, __nv_bfloat16>(a, s); }

}  // namespace qgemv
