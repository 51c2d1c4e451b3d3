// ddt_gqa_chunk_cap.cu -- chunk attention and received weights with capped scores.
#include "ddt_gqa_chunk_attn.cuh"
#include "ddt_gqa_chunk_weights.cuh"

namespace ddt {
namespace chunk {
template cudaError_t launch_attn_score<1>(AttnParams &prm, cudaStream_t s);
template cudaError_t prepare_attn_score<1>();
namespace received {
template cudaError_t launch_weights_score<1>(Params &prm, int nq, cudaStream_t s);
template cudaError_t prepare_weights_score<1>();
}  // namespace received
}  // namespace chunk
}  // namespace ddt
