// ddt_gqa_chunk_bias.cu -- chunk attention with scores with a distance bias.
#include "ddt_gqa_chunk_attn.cuh"

namespace ddt {
namespace chunk {
template cudaError_t launch_attn_score<2>(AttnParams &prm, cudaStream_t s);
template cudaError_t prepare_attn_score<2>();
}  // namespace chunk
}  // namespace ddt
