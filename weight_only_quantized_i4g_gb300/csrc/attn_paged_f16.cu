// attn_paged_f16.cu -- the attention kernels over an f16 cache.
#include "attn_launch.cuh"

namespace qg {
template int launch_attn_stream<kF16, false>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2], cudaStream_t);
template AttnPlan attn_plan<kF16>(int rows, int dim);
}
