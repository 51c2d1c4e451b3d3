// ddt_gqa_chunk_plain.cu -- chunk attention with plain scores.
#include "ddt_gqa_chunk_attn.cuh"

namespace ddt {
namespace chunk {
template cudaError_t launch_attn_score<0>(AttnParams &prm, cudaStream_t s);
template cudaError_t prepare_attn_score<0>();
}  // namespace chunk
}  // namespace ddt
