// ddt_gqa_chunk_cap_bias.cu -- chunk attention and received weights with capped scores with a distance bias.
#include "ddt_gqa_chunk_attn.cuh"
#include "ddt_gqa_chunk_weights.cuh"

namespace ddt {
namespace chunk {
template cudaError_t launch_attn_score<3>(AttnParams &prm, cudaStream_t s);
template cudaError_t prepare_attn_score<3>();
namespace received {
template cudaError_t launch_weights_score<3>(Params &prm, int nq, cudaStream_t s);
template cudaError_t prepare_weights_score<3>();
}  // namespace received
}  // namespace chunk
}  // namespace ddt
