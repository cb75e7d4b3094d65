// attn_paged over q8_0 pages for bf16 rows.
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_q8_0_bf16(const AttnArgs& a, cudaStream_t s) { return launch_attn_rows<QGEMV_KV_Q8_0, __nv_bfloat16>(a, s); }

}  // namespace qgemv
