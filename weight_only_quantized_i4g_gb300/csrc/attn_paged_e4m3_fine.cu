// attn_paged_e4m3_fine.cu -- the attention kernels over an e4m3 cache, f32 or f16 output.
#include "attn_launch.cuh"

namespace qg {
template int launch_attn_stream<kE4m3, true>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2], cudaStream_t);
}
