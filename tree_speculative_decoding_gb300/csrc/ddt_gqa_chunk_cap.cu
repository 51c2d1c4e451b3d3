// ddt_gqa_chunk_cap.cu -- chunk attention with capped scores.
#include "ddt_gqa_chunk_attn.cuh"

namespace ddt {
namespace chunk {
template cudaError_t launch_attn_score<1>(AttnParams &prm, cudaStream_t s);
template cudaError_t prepare_attn_score<1>();
}  // namespace chunk
}  // namespace ddt
