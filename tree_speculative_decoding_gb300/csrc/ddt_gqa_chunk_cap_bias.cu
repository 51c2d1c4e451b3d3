// ddt_gqa_chunk_cap_bias.cu -- chunk attention with capped scores with a distance bias.
#include "ddt_gqa_chunk_attn.cuh"

namespace ddt {
namespace chunk {
template cudaError_t launch_attn_score<3>(AttnParams &prm, cudaStream_t s);
template cudaError_t prepare_attn_score<3>();
}  // namespace chunk
}  // namespace ddt
