// attn_paged over f16 pages.
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_f16(int type, const AttnArgs& a, cudaStream_t s) { return launch_attn_type<QGEMV_KV_F16>(type, a, s); }

}  // namespace qgemv
