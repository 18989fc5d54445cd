// zdmmv_attn_d256.cu -- the attention kernels for heads of 256 dimensions.
#define ZDMMV_ATTN_INSTANTIATE
#include "zdmmv_attn.cuh"

namespace zdmmv {
template cudaError_t launch_attn<8>(AttnArgs, const AttnPlan &, cudaStream_t);
}  // namespace zdmmv
