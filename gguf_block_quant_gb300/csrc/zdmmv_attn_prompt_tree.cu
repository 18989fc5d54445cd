// zdmmv_attn_prompt_tree.cu -- the attention kernels with a tree's order and lse of many columns, heads of 64, 96 and 128 dimensions.
#include "zdmmv_attn_prompt.cuh"

namespace zdmmv {
template cudaError_t launch_attn_tall<2, true>(const AttnArgs &, const AttnPlan &, cudaStream_t);
template cudaError_t launch_attn_tall<3, true>(const AttnArgs &, const AttnPlan &, cudaStream_t);
template cudaError_t launch_attn_tall<4, true>(const AttnArgs &, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
