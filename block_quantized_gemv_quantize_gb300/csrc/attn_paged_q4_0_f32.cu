// attn_paged over q4_0 pages for f32 rows.
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_q4_0_f32(const AttnArgs& a, cudaStream_t s) { return launch_attn_rows<QGEMV_KV_Q4_0, float>(a, s); }

}  // namespace qgemv
