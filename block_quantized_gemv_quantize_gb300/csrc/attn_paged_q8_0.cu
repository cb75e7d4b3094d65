// attn_paged over q8_0 pages.
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_q8_0(int type, const AttnArgs& a, cudaStream_t s) { return launch_attn_type<QGEMV_KV_Q8_0>(type, a, s); }

}  // namespace qgemv
