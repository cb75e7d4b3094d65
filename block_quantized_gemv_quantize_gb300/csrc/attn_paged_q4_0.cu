// attn_paged over q4_0 pages.
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_q4_0(int type, const AttnArgs& a, cudaStream_t s) { return launch_attn_type<QGEMV_KV_Q4_0>(type, a, s); }

}  // namespace qgemv
