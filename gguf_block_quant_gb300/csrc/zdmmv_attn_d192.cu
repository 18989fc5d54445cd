// zdmmv_attn_d192.cu -- the attention kernels for heads of 192 dimensions.
#define ZDMMV_ATTN_INSTANTIATE
#include "zdmmv_attn.cuh"

namespace zdmmv {
template cudaError_t launch_attn<6, false>(AttnArgs, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
