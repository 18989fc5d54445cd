// zdmmv_attn_tree_d64.cu -- the attention kernels with a tree's order and lse for heads of 64 dimensions.
#define ZDMMV_ATTN_INSTANTIATE
#include "zdmmv_attn.cuh"

namespace zdmmv {
template cudaError_t launch_attn<2, true>(AttnArgs, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
