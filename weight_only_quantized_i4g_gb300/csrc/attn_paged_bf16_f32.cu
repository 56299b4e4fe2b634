// attn_paged_bf16_f32.cu -- the attention kernels over a bf16 cache, f32 or f16 output.
#include "attn_launch.cuh"

namespace qg {
template int launch_attn_stream<kBf16, true>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2], cudaStream_t);
}
