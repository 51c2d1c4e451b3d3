// ddt_gqa_chunk_plain.cu -- chunk attention and received weights with plain scores.
#include "ddt_gqa_chunk_attn.cuh"
#include "ddt_gqa_chunk_weights.cuh"

namespace ddt {
namespace chunk {
template cudaError_t launch_attn_score<0>(AttnParams &prm, cudaStream_t s);
template cudaError_t prepare_attn_score<0>();
namespace received {
template cudaError_t launch_weights_score<0>(Params &prm, int nq, cudaStream_t s);
template cudaError_t prepare_weights_score<0>();
}  // namespace received
}  // namespace chunk
}  // namespace ddt
