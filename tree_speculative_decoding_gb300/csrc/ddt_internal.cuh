// ddt_internal.cuh -- declarations shared by the CUDA translation units of
// libddt.so (launchers defined in each .cu, called from ddt_abi.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ddt.h"

namespace ddt {

// Latch a device-side check into the per-device error word.
__device__ __forceinline__ void latch(unsigned int *err, unsigned int bit) {
    if (err) atomicOr(err, bit);
}

// Programmatic dependent launch.  Every kernel of the library is launched with
// programmatic stream serialization and announces at its start that the next
// kernel in the stream may be scheduled.  A kernel therefore may run while the
// previous one is still running, and it calls pdl_wait() -- which returns once
// the previous kernel (and, transitively, everything before it) has finished
// and its writes are visible -- before it reads anything an earlier kernel of
// the step wrote, and before its first global write.  Work on the caller's
// inputs (q, the kv pool and indices, top-k) may happen before the wait; a
// kernel that does not itself trigger early is complete before any of ours
// starts.  Dependents are scheduled only after every CTA of the previous
// kernel has started, so no wait can hold resources the previous kernel needs.
__device__ __forceinline__ void pdl_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Launchers (host functions; each enqueues on `s` and returns the launch error).
cudaError_t launch_build_tree(const float *topk_logp, const int32_t *topk_ids,
                              const int32_t *root_id, const int32_t *budget,
                              const int32_t *qo_indptr, int batch, int max_depth, int topk,
                              int32_t *node_token, int32_t *parent, int32_t *depth,
                              unsigned int *err, cudaStream_t s);

cudaError_t launch_build_tree_visibility(const float *topk_logp, const int32_t *topk_ids,
                                         const int32_t *root_id, const int32_t *budget,
                                         const int32_t *qo_indptr, int batch, int max_depth, int topk,
                                         const int32_t *prefix_len, const int32_t *mask_indptr,
                                         int32_t *node_token, int32_t *parent, int32_t *depth,
                                         uint32_t *mask, unsigned int *err, cudaStream_t s);
cudaError_t launch_build_chain_visibility(const int32_t *qo_indptr, const int32_t *prefix_len,
                                          const int32_t *mask_indptr, int batch, int32_t *parent,
                                          int32_t *depth, uint32_t *mask, unsigned int *err,
                                          cudaStream_t s);
cudaError_t launch_compile_visibility(const int32_t *parent, const int32_t *qo_indptr,
                                      const int32_t *prefix_len, const int32_t *mask_indptr,
                                      int batch, int total_words, uint32_t *mask,
                                      unsigned int *err, cudaStream_t s);

cudaError_t launch_accept(const int32_t *node_token, const int32_t *parent,
                          const int32_t *qo_indptr, const int32_t *target_argmax, int batch,
                          int max_depth, int32_t *accept_len, int32_t *accepted_nodes,
                          int32_t *commit_tokens, int32_t *bonus, unsigned int *err,
                          cudaStream_t s);

cudaError_t launch_commit_kv(uint16_t *kv_pool, int64_t pool_rows, const int32_t *kv_indices,
                             const int32_t *kv_indptr, const int32_t *qo_indptr,
                             const int32_t *accept_len, const int32_t *accepted_nodes, int batch,
                             int max_depth, int32_t *new_len, unsigned int *err, cudaStream_t s);

cudaError_t launch_tree_links(const int32_t *parent, const int32_t *qo_indptr, int batch,
                              int32_t *first_child, int32_t *next_sibling, int32_t *retrieve_index,
                              unsigned int *err, cudaStream_t s);
cudaError_t launch_accept_sampled(const int32_t *node_token, const int32_t *first_child,
                                  const int32_t *next_sibling, const int32_t *qo_indptr,
                                  const float *logits, int vocab, const float *temperature,
                                  const int32_t *top_k, const float *top_p, const float *coins,
                                  int coin_stride, int batch,
                                  int max_depth, int32_t *accept_len, int32_t *accepted_nodes,
                                  int32_t *commit_tokens, int32_t *bonus, unsigned int *err,
                                  cudaStream_t s);

// Arguments of one verify-attention call as seen by the kernels.
struct AttnArgs {
    const uint16_t *q;
    const uint16_t *kv_pool;
    int64_t pool_rows;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    const int32_t *qo_indptr;
    const uint32_t *mask;
    const int32_t *mask_indptr;
    int batch;
    int num_heads;
    int total_q;
    int max_q_len;
    int max_kv_len;
    float scale;
    int num_splits;
    int split_cols;       // kv columns per split (multiple of the kv tile)
    // 1 when the mask is a tree mask this library built in the same step (every
    // prefix column visible, no column after the row's own node): prefix-only
    // blocks then read no mask word.  0: every mask bit is honoured.
    int tree_mask;
    float *out;           // [total_q, H, 512]
    float *lse;           // [total_q, H] or null
    float *o_part;        // [splits, total_q*H, 512] when num_splits > 1
    float *lse_part;      // [splits, total_q*H]
    unsigned int *err;
};

// Split-KV partial pass (tensor-core kernel) and its sizing rules.
cudaError_t launch_attn_partial(const AttnArgs &a, cudaStream_t s);
// the split count for these bounds, at most max_splits (>= 1)
int attn_choose_splits(int batch, int num_heads, int max_q_len, int max_kv_len, int num_sms,
                       int max_splits = DDT_MAX_SPLITS);
cudaError_t attn_tc_prepare_device();
// CUDA-core kernel of the same pass (same arguments and outputs)
cudaError_t launch_attn_combine(const AttnArgs &a, cudaStream_t s);
cudaError_t attn_combine_prepare_device();
// shared-memory carveout of the small stages' kernels (they overlap the attention)
cudaError_t tree_prepare_device();
cudaError_t commit_prepare_device();
cudaError_t sample_prepare_device();

// Arguments of one norm + rotation + append call as seen by the kernel.
struct AppendArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements per token
    const uint16_t *q_weight, *k_weight;   // or null
    float eps;
    const float *cos_sin;  // [max_pos][rope_dim]: cosines, then sines
    int64_t max_pos;
    int rope_dim;
    int interleaved;
    const int32_t *depth;  // or null: the token's index in its request
    const int32_t *qo_indptr;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    int batch;
    int total_q;
    int total_kv;
    int num_heads;
    int num_kv_heads;
    int head_dim;
    uint16_t *q_out;
    uint16_t *k_pool, *v_pool;
    int64_t pool_stride;  // elements per row
    int64_t pool_rows;
    unsigned int *err;
};
cudaError_t launch_norm_rope_append(const AppendArgs &a, int num_sms, cudaStream_t s);

// Arguments of one grouped-query attention call as seen by the kernels.
struct GqaArgs {
    const uint16_t *q;
    const uint16_t *k_pool, *v_pool;
    int64_t pool_stride;  // elements per row
    int64_t pool_rows;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    const int32_t *qo_indptr;
    const uint32_t *mask;
    const int32_t *mask_indptr;
    int batch;
    int num_heads;
    int num_kv_heads;
    int head_dim;
    int total_q;
    int total_kv;
    int total_mask_words;
    int max_q_len;
    int max_kv_len;
    float scale;
    // CTAs that the blocks of columns are dealt to (batch <= kGqaMaxDealtBatch),
    // or 0: one CTA per item, no workspace
    int num_ctas;
    int forced;       // the caller gave the count: a CTA may get a single block
    int tiles;        // tiles of 128 rows of an item: 1 or 2
    uint16_t *out;    // [total_q, H, D] bf16
    float *lse;       // [total_q, H] or null
    // dealt: per item the place of its first part (-1: whole) and the CTA with its last
    int2 *notes;      // [batch][num_kv_heads][gqa_tile_groups()]
    float *o_part;    // [2 * num_ctas][gqa_part_rows()][D]
    float *lse_part;  // [2 * num_ctas][gqa_part_rows()]
    unsigned int *err;
};
constexpr int kGqaMaxDealtBatch = 256;  // a thread per request sizes the line
// kernel attributes, once per device (see attn_prepare_device)
cudaError_t gqa_prepare_device();
cudaError_t launch_gqa_attn(const GqaArgs &a, int num_sms, cudaStream_t s);
// the most CTAs that the work may be dealt to for these bounds, or 0 (see GqaArgs)
int gqa_most_ctas(int batch, int num_heads, int num_kv_heads, int max_q_len, int max_kv_len, int num_sms);
// tiles of an item where the caller gives the count of CTAs
int gqa_tiles(int max_q_len, int group);
// a.tiles and a.num_ctas for the call's sizes, within the workspace
void gqa_choose(GqaArgs &a, size_t workspace_bytes, int num_sms);
// rows of a partial result; most items per K/V head of a request
int gqa_part_rows(int tiles, int max_q_len, int group);
int gqa_tile_groups(int tiles, int max_q_len, int group);
// bytes of the workspace for a.tiles and a.num_ctas; places its parts in a where base is given
size_t gqa_layout(GqaArgs &a, void *base);

// Arguments of one chunk call (attention or received weights) as seen by the kernels.
struct ChunkArgs {
    const uint16_t *q;
    const uint16_t *k_pool, *v_pool;
    int64_t pool_stride;  // elements per row
    int64_t pool_rows;
    const int32_t *kv_indices;
    const int32_t *kv_indptr;
    const int32_t *qo_indptr;
    int batch;
    int num_heads;
    int num_kv_heads;
    int head_dim;
    int total_q;
    int total_kv;
    int max_q_len;
    int max_kv_len;
    float scale;
    float score_cap;       // 0: none
    const float *slopes;   // [num_heads] or null
    int window;            // 0: none
    const int32_t *full_len;  // [batch] or null
    // attention
    int num_ctas;     // CTAs that the blocks of columns are dealt to, or 0: one CTA per item
    int forced;       // the caller gave the count: a CTA may get a single block
    int tiles;        // tiles of 128 rows of an item: 1 or 2
    uint16_t *out;    // [total_q, H, D] bf16
    float *lse;       // [total_q, H]: out (or null) of the attention, input of the weights
    int4 *notes;      // [num_ctas]: the cut item that ends in a CTA's share
    float *o_part;    // [2 * num_ctas][part rows][D]
    float *lse_part;  // [2 * num_ctas][part rows]
    unsigned int *err;
};
// What a received-weights call has besides (in ChunkArgs: o_part [2 * num_ctas][256]).
struct WeightArgs {
    int last_rows;              // tokens of a request that count, from its end; 0: all
    const float *prev;          // or null
    const int32_t *prev_indptr; // or null: kv_indptr
    int total_prev;
    float decay;
    float *weights;             // [total_kv]
};
constexpr int kChunkMaxDealtBatch = 256;  // a thread per request places it on the line
cudaError_t chunk_prepare_device();
cudaError_t launch_chunk_attn(const ChunkArgs &a, int num_sms, cudaStream_t s);
// the most CTAs that the work may be dealt to for these bounds, or 0
int chunk_most_ctas(int batch, int num_heads, int num_kv_heads, int max_q_len, int max_kv_len, int num_sms);
int chunk_tiles(int max_q_len, int group);
// a.tiles and a.num_ctas for the call's sizes, within the workspace
void chunk_choose(ChunkArgs &a, size_t workspace_bytes, int num_sms);
cudaError_t launch_chunk_weights(const ChunkArgs &a, const WeightArgs &w, cudaStream_t s);
int chunk_weights_most_ctas(int batch, int num_sms);
size_t chunk_weights_layout(ChunkArgs &a, void *base);
// bytes of the workspace for a.tiles and a.num_ctas; places its parts in a where base is given
size_t chunk_layout(ChunkArgs &a, void *base);

// Arguments of an eviction as seen by the kernel.
struct EvictArgs {
    const float *weights;        // [total_kv]
    const int32_t *kv_indices;   // [total_kv]
    const int32_t *kv_indptr;
    const int32_t *budget;       // [batch]
    int batch;
    int total_kv;
    int max_kv_len;
    int sinks, recent;
    int32_t *new_indices;        // [total_new]
    int total_new;
    int32_t *new_indptr;         // [batch + 1]
    float *new_weights;          // [total_new] or null
    int32_t *evicted;            // [total_evicted] or null
    int total_evicted;
    unsigned int *err;
};
cudaError_t evict_prepare_device();
cudaError_t launch_cache_evict(const EvictArgs &a, cudaStream_t s);

cudaError_t launch_cache_copy(const void *src_slab, int64_t src_pool_bytes, int64_t src_rows, void *dst_slab,
                              int64_t dst_pool_bytes, int64_t dst_rows, int num_pools, int64_t row_bytes,
                              const int32_t *src, const int32_t *dst, int n, unsigned int *err, cudaStream_t s);
cudaError_t launch_cache_commit(void *slab, int64_t pool_bytes, int64_t pool_rows, int num_pools, int64_t row_bytes,
                                const int32_t *kv_indices, const int32_t *kv_indptr, const int32_t *qo_indptr,
                                const int32_t *accept_len, const int32_t *accepted_nodes, int batch, int total_kv,
                                int max_depth, int32_t *new_len, int num_sms, unsigned int *err, cudaStream_t s);
size_t cache_compact_workspace(int64_t pool_rows);
cudaError_t launch_cache_compact(void *slab, int64_t pool_bytes, int64_t pool_rows, int num_pools, int64_t row_bytes,
                                 const int32_t *kv_indices, int total, int32_t *new_indices, int32_t *live,
                                 void *workspace, int num_sms, unsigned int *err, cudaStream_t s);

// A kernel whose bounded mbarrier wait can never succeed: it latches
// DDT_DEVERR_TIMEOUT and exits (the failure path, exercised without a fault).
cudaError_t launch_wait_timeout_selftest(uint32_t poll_limit, unsigned int *err, cudaStream_t s);

// kv columns per split must be a multiple of this (the attention kv tile)
int attn_kv_tile();
// The split layout a requested count (>= 1) gives: kv columns per split,
// rounded up to whole kv tiles, and the number of splits that then cover
// max_kv_len (no empty tail split), which can be fewer than requested.
void attn_split_layout(int max_kv_len, int requested, int *split_cols, int *splits);
int attn_launched_splits(int max_kv_len, int requested);

// Once per device, with that device current and before any stream capture:
// kernel attributes (dynamic shared memory opt-in).
cudaError_t attn_prepare_device();

// Device address of the current device's error word (null on failure).
unsigned int *device_error_word();
// the current device's SM count (after the same one-time set-up)
int device_sm_count();

}  // namespace ddt
