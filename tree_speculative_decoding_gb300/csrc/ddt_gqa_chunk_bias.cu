// ddt_gqa_chunk_bias.cu -- chunk attention and received weights with scores with a distance bias.
#include "ddt_gqa_chunk_attn.cuh"
#include "ddt_gqa_chunk_weights.cuh"

namespace ddt {
namespace chunk {
template cudaError_t launch_attn_score<2>(AttnParams &prm, cudaStream_t s);
template cudaError_t prepare_attn_score<2>();
namespace received {
template cudaError_t launch_weights_score<2>(Params &prm, int nq, cudaStream_t s);
template cudaError_t prepare_weights_score<2>();
}  // namespace received
}  // namespace chunk
}  // namespace ddt
