// zdmmv_attn_prompt.cu -- the prompts' attention kernels for heads of 64, 96 and 128 dimensions.
#include "zdmmv_attn_prompt.cuh"

namespace zdmmv {
template cudaError_t launch_attn_prompt<2>(const AttnArgs &, const AttnPlan &, cudaStream_t);
template cudaError_t launch_attn_prompt<3>(const AttnArgs &, const AttnPlan &, cudaStream_t);
template cudaError_t launch_attn_prompt<4>(const AttnArgs &, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
