// attn_paged over q4_0 pages for f16 rows.
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_q4_0_f16(const AttnArgs& a, cudaStream_t s) { return launch_attn_rows<QGEMV_KV_Q4_0, __half>(a, s); }

}  // namespace qgemv
