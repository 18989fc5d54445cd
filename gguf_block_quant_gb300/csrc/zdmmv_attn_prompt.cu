// zdmmv_attn_prompt.cu -- the attention kernels of many columns, heads of 64, 96 and 128 dimensions.
#include "zdmmv_attn_prompt.cuh"

namespace zdmmv {
template cudaError_t launch_attn_tall<2, false>(const AttnArgs &, const AttnPlan &, cudaStream_t);
template cudaError_t launch_attn_tall<3, false>(const AttnArgs &, const AttnPlan &, cudaStream_t);
template cudaError_t launch_attn_tall<4, false>(const AttnArgs &, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
