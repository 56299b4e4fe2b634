// attn_paged_bf16.cu -- the attention kernels over a bf16 cache, bf16 output.
#include "attn_launch.cuh"

namespace qg {
template int launch_attn_stream<kBf16, false>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2], cudaStream_t);
template AttnPlan attn_plan<kBf16>(int rows, int dim);
}
