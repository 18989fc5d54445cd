// zdmmv_attn_d64.cu -- the attention kernels for heads of 64 dimensions.
#define ZDMMV_ATTN_INSTANTIATE
#include "zdmmv_attn.cuh"

namespace zdmmv {
template cudaError_t launch_attn<2, false>(AttnArgs, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
