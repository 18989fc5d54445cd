// zdmmv_attn_d96.cu -- the attention kernels for heads of 96 dimensions.
#define ZDMMV_ATTN_INSTANTIATE
#include "zdmmv_attn.cuh"

namespace zdmmv {
template cudaError_t launch_attn<3>(AttnArgs, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
