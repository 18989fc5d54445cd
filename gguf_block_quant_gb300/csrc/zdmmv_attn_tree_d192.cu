// zdmmv_attn_tree_d192.cu -- the attention kernels with a tree's order and lse for heads of 192 dimensions.
#define ZDMMV_ATTN_INSTANTIATE
#include "zdmmv_attn.cuh"

namespace zdmmv {
template cudaError_t launch_attn<6, true>(AttnArgs, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
