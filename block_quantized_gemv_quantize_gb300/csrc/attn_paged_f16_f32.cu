// attn_paged over f16 pages for f32 rows.
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_f16_f32(const AttnArgs& a, cudaStream_t s) { return launch_attn_rows<QGEMV_KV_F16, float>(a, s); }

}  // namespace qgemv
