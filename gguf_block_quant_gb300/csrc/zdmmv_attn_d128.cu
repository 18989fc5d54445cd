// zdmmv_attn_d128.cu -- the attention kernels for heads of 128 dimensions.
#define ZDMMV_ATTN_INSTANTIATE
#include "zdmmv_attn.cuh"

namespace zdmmv {
template cudaError_t launch_attn<4, false>(AttnArgs, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
