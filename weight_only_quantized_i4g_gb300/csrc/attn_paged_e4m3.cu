// attn_paged_e4m3.cu -- the attention kernels over an e4m3 cache, bf16 output.
#include "attn_launch.cuh"

namespace qg {
template int launch_attn_stream<kE4m3, false>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2], cudaStream_t);
template AttnPlan attn_plan<kE4m3>(int rows, int dim);
}
