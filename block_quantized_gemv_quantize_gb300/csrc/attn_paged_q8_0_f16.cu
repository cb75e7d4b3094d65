// attn_paged over q8_0 pages for f16 rows.
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_q8_0_f16(const AttnArgs& a, cudaStream_t s) { return launch_attn_rows<QGEMV_KV_Q8_0, __half>(a, s); }

}  // namespace qgemv
