// ddt_gqa_abi.cu -- the extern "C" entry points of the grouped-query layer and
// of the cache-row calls: host-side argument checks, sizing and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>
#include <utility>

#include "ddt_internal.cuh"

namespace {

inline cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }
inline bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
inline ddt_status launched(cudaError_t e) { return e == cudaSuccess ? DDT_OK : DDT_ERR_CUDA; }

// head layout of a grouped-query call
ddt_status check_heads(int32_t num_heads, int32_t num_kv_heads, int32_t head_dim) {
    if (num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads) return DDT_ERR_INVALID_ARG;
    if (num_heads > DDT_GQA_MAX_HEADS || (head_dim != 64 && head_dim != 128)) return DDT_ERR_UNSUPPORTED;
    return DDT_OK;
}
bool bad_pool_stride(int64_t stride, int32_t num_kv_heads, int32_t head_dim) {
    return stride < (int64_t)num_kv_heads * head_dim || stride % 8;
}

// whether a[0 .. na) and b[0 .. nb) share a byte
template <class T, class U>
bool overlap(const T *a, int64_t na, const U *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && (x < y ? (y - x) / sizeof(T) < (uint64_t)na : (x - y) / sizeof(U) < (uint64_t)nb);
}
// elements from the first row's start to the last row's end
int64_t extent(int32_t rows, int64_t stride, int64_t width) { return (rows - 1) * stride + width; }

// columns of a request that are counted in 32 bits, with a block behind them
constexpr int32_t kMostColumns = INT32_MAX - 127;

// layout of a slab of pools
bool bad_slab(const void *slab, int64_t pool_bytes, int64_t pool_rows, int32_t num_pools, int64_t row_bytes) {
    if (!slab || misaligned(slab, 16) || pool_rows < 1 || num_pools < 1 || row_bytes < 16 || row_bytes % 16 ||
        pool_bytes % 16 || row_bytes / 16 > INT32_MAX)
        return true;
    return pool_rows > INT64_MAX / row_bytes || pool_bytes < pool_rows * row_bytes;
}

// a parameter of type T from its word; fits: false where it does not hold the word's value
template <class T>
T from_word(int64_t w, bool &fits) {
    if constexpr (std::is_pointer_v<T>) {
        return reinterpret_cast<T>((uintptr_t)w);
    } else if constexpr (std::is_floating_point_v<T>) {
        double d;
        memcpy(&d, &w, sizeof d);
        return (T)d;
    } else {
        fits = fits && (int64_t)(T)w == w;
        return (T)w;
    }
}
template <class... A, size_t... I>
ddt_status call_with(ddt_status (*f)(A...), const int64_t *words, std::index_sequence<I...>) {
    bool fits = words[1] == (int64_t)sizeof...(A);
    if (!fits) return DDT_ERR_INVALID_ARG;
    const auto go = [&](A... a) { return fits ? f(a...) : DDT_ERR_INVALID_ARG; };
    return go(from_word<A>(words[2 + I], fits)...);
}
template <class... A>
ddt_status call_words(ddt_status (*f)(A...), const int64_t *words) {
    return call_with(f, words, std::index_sequence_for<A...>{});
}

}  // namespace

extern "C" {

ddt_status ddt_gqa_norm_rope_append(
    const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride, const uint16_t *v,
    int64_t v_stride, const uint16_t *q_weight, const uint16_t *k_weight, float eps,
    const float *cos_sin, int64_t max_pos, int32_t rope_dim, int32_t interleaved,
    const int32_t *depth, const int32_t *qo_indptr, const int32_t *kv_indices,
    const int32_t *kv_indptr, int32_t batch, int32_t total_q, int32_t total_kv, int32_t num_heads,
    int32_t num_kv_heads, int32_t head_dim, uint16_t *q_out, uint16_t *k_pool, uint16_t *v_pool,
    int64_t pool_stride, int64_t pool_rows, void *stream) {
    if (!q || !k || !v || !qo_indptr || (!kv_indices && total_kv != 0) || !kv_indptr || !q_out || !k_pool ||
        !v_pool || batch < 0 || total_q < 0 || total_kv < 0 || pool_rows < 1 || !(eps >= 0.f) || !isfinite(eps) || rope_dim < 0 || max_pos < 0 ||
        (rope_dim > 0 && !cos_sin))
        return DDT_ERR_INVALID_ARG;
    const ddt_status heads = check_heads(num_heads, num_kv_heads, head_dim);
    if (heads != DDT_OK) return heads;
    if (rope_dim % 16 || rope_dim > head_dim) return DDT_ERR_UNSUPPORTED;
    const int64_t qw = (int64_t)num_heads * head_dim, kw = (int64_t)num_kv_heads * head_dim;
    if (q_stride < qw || k_stride < kw || v_stride < kw || q_stride % 8 || k_stride % 8 || v_stride % 8 ||
        bad_pool_stride(pool_stride, num_kv_heads, head_dim))
        return DDT_ERR_INVALID_ARG;
    // in place only where a token's rows stay where they are
    if (q_out == q && q_stride != qw) return DDT_ERR_INVALID_ARG;
    const void *aligned[] = {q, k, v, q_weight, k_weight, cos_sin, q_out, k_pool, v_pool};
    for (const void *p : aligned)
        if (misaligned(p, 16)) return DDT_ERR_INVALID_ARG;
    if (batch == 0 || total_q == 0) return DDT_OK;
    // what a token reads may not be what another one writes
    const int64_t q_out_size = extent(total_q, qw, qw);
    if ((q_out != q && overlap(q_out, q_out_size, q, extent(total_q, q_stride, qw))) ||
        overlap(q_out, q_out_size, k, extent(total_q, k_stride, kw)) ||
        overlap(q_out, q_out_size, v, extent(total_q, v_stride, kw)))
        return DDT_ERR_INVALID_ARG;
    unsigned int *err = ddt::device_error_word();
    if (!err) return DDT_ERR_CUDA;
    ddt::AppendArgs a;
    memset(&a, 0, sizeof a);
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.cos_sin = cos_sin;
    a.max_pos = max_pos;
    a.rope_dim = rope_dim;
    a.interleaved = interleaved != 0;
    a.depth = depth;
    a.qo_indptr = qo_indptr;
    a.kv_indices = kv_indices;
    a.kv_indptr = kv_indptr;
    a.batch = batch;
    a.total_q = total_q;
    a.total_kv = total_kv;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.q_out = q_out;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.pool_stride = pool_stride;
    a.pool_rows = pool_rows;
    a.err = err;
    return launched(ddt::launch_norm_rope_append(a, ddt::device_sm_count(), as_stream(stream)));
}

int32_t ddt_gqa_verify_attn_num_ctas(int32_t batch, int32_t num_heads, int32_t num_kv_heads,
                                     int32_t max_q_len, int32_t max_kv_len, int32_t num_sms) {
    if (batch < 1 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads || max_q_len < 1 ||
        max_kv_len < 1)
        return 0;
    if (num_sms <= 0) num_sms = ddt::device_sm_count();
    return ddt::gqa_most_ctas(batch, num_heads, num_kv_heads, max_q_len, max_kv_len, num_sms);
}

size_t ddt_gqa_verify_attn_workspace_size(int32_t batch, int32_t num_heads, int32_t num_kv_heads,
                                          int32_t head_dim, int32_t max_q_len, int32_t num_ctas) {
    if (batch < 1 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads || head_dim < 1 || max_q_len < 1 ||
        num_ctas < 1)
        return 0;
    ddt::GqaArgs a;
    memset(&a, 0, sizeof a);
    a.batch = batch;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.max_q_len = max_q_len;
    a.tiles = ddt::gqa_tiles(max_q_len, num_heads / num_kv_heads);
    a.num_ctas = num_ctas;
    size_t bytes = ddt::gqa_layout(a, nullptr);
    if (a.tiles == 2) {  // num_ctas = 0 may take one tile and twice as many CTAs instead
        a.tiles = 1;
        a.num_ctas = 2 * num_ctas;
        const size_t other = ddt::gqa_layout(a, nullptr);
        if (other > bytes) bytes = other;
    }
    return bytes;
}

ddt_status ddt_gqa_verify_attn(
    const uint16_t *q, const uint16_t *k_pool, const uint16_t *v_pool, int64_t pool_stride,
    int64_t pool_rows, const int32_t *kv_indices, const int32_t *kv_indptr,
    const int32_t *qo_indptr, const uint32_t *mask, const int32_t *mask_indptr, int32_t batch,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t total_q, int32_t total_kv,
    int32_t total_mask_words, int32_t max_q_len, int32_t max_kv_len, float scale,
    int32_t num_ctas, uint16_t *out, float *lse, void *workspace, size_t workspace_bytes,
    void *stream) {
    if (!q || !k_pool || !v_pool || (!kv_indices && total_kv != 0) || !kv_indptr || !qo_indptr ||
        (!mask && total_mask_words != 0) || !mask_indptr || !out || batch < 0 || total_q < 0 || total_kv < 0 ||
        total_mask_words < 0 || pool_rows < 1 || max_q_len < 0 || max_kv_len < max_q_len || !isfinite(scale) || !(scale > 0.f) || num_ctas < 0)
        return DDT_ERR_INVALID_ARG;
    const ddt_status heads = check_heads(num_heads, num_kv_heads, head_dim);
    if (heads != DDT_OK) return heads;
    if (max_q_len > DDT_MAX_Q_LEN || num_ctas > DDT_GQA_MAX_CTAS || pool_rows > INT32_MAX || batch > 65535 ||
        (num_ctas > 0 && batch > ddt::kGqaMaxDealtBatch))
        return DDT_ERR_UNSUPPORTED;
    if (misaligned(q, 16) || misaligned(k_pool, 16) || misaligned(v_pool, 16) || misaligned(out, 16) ||
        misaligned(workspace, 256) || bad_pool_stride(pool_stride, num_kv_heads, head_dim))
        return DDT_ERR_INVALID_ARG;
    if (batch == 0 || total_q == 0 || max_q_len == 0) return DDT_OK;
    // CTAs that share an item read its q, one maybe after another's output
    const int64_t rows_size = (int64_t)total_q * num_heads * head_dim;
    if (overlap(out, rows_size, q, rows_size)) return DDT_ERR_INVALID_ARG;
    unsigned int *err = ddt::device_error_word();
    if (!err) return DDT_ERR_CUDA;

    ddt::GqaArgs a;
    memset(&a, 0, sizeof a);
    a.q = q;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.pool_stride = pool_stride;
    a.pool_rows = pool_rows;
    a.kv_indices = kv_indices;
    a.kv_indptr = kv_indptr;
    a.qo_indptr = qo_indptr;
    a.mask = mask;
    a.mask_indptr = mask_indptr;
    a.batch = batch;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.total_q = total_q;
    a.total_kv = total_kv;
    a.total_mask_words = total_mask_words;
    a.max_q_len = max_q_len;
    a.max_kv_len = max_kv_len < kMostColumns ? max_kv_len : kMostColumns;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.err = err;
    const int num_sms = ddt::device_sm_count();
    if (num_ctas > 0) {
        a.forced = 1;
        a.tiles = ddt::gqa_tiles(max_q_len, num_heads / num_kv_heads);
        a.num_ctas = num_ctas;
        if (!workspace || workspace_bytes < ddt::gqa_layout(a, nullptr)) return DDT_ERR_WORKSPACE;
    } else {
        ddt::gqa_choose(a, workspace ? workspace_bytes : 0, num_sms);
    }
    if (a.num_ctas > 0) ddt::gqa_layout(a, workspace);
    return launched(ddt::launch_gqa_attn(a, num_sms, as_stream(stream)));
}

ddt_status ddt_cache_copy(const void *src_slab, int64_t src_pool_bytes, int64_t src_pool_rows,
                          void *dst_slab, int64_t dst_pool_bytes, int64_t dst_pool_rows,
                          int32_t num_pools, int64_t row_bytes, const int32_t *src,
                          const int32_t *dst, int32_t n, void *stream) {
    if (bad_slab(src_slab, src_pool_bytes, src_pool_rows, num_pools, row_bytes) ||
        bad_slab(dst_slab, dst_pool_bytes, dst_pool_rows, num_pools, row_bytes) || n < 0 || (n > 0 && (!src || !dst)))
        return DDT_ERR_INVALID_ARG;
    if (n == 0) return DDT_OK;
    unsigned int *err = ddt::device_error_word();
    if (!err) return DDT_ERR_CUDA;
    return launched(ddt::launch_cache_copy(src_slab, src_pool_bytes, src_pool_rows, dst_slab, dst_pool_bytes,
                                           dst_pool_rows, num_pools, row_bytes, src, dst, n, err, as_stream(stream)));
}

ddt_status ddt_cache_commit(void *slab, int64_t pool_bytes, int64_t pool_rows, int32_t num_pools,
                            int64_t row_bytes, const int32_t *kv_indices, const int32_t *kv_indptr,
                            const int32_t *qo_indptr, const int32_t *accept_len,
                            const int32_t *accepted_nodes, int32_t batch, int32_t total_kv,
                            int32_t max_depth, int32_t *new_len, void *stream) {
    if (bad_slab(slab, pool_bytes, pool_rows, num_pools, row_bytes) || (!kv_indices && total_kv != 0) || !kv_indptr ||
        !qo_indptr || !accept_len || !accepted_nodes || batch < 0 || total_kv < 0)
        return DDT_ERR_INVALID_ARG;
    if (max_depth < 1 || max_depth > DDT_MAX_DEPTH) return DDT_ERR_UNSUPPORTED;
    if (batch == 0) return DDT_OK;
    unsigned int *err = ddt::device_error_word();
    if (!err) return DDT_ERR_CUDA;
    return launched(ddt::launch_cache_commit(slab, pool_bytes, pool_rows, num_pools, row_bytes, kv_indices, kv_indptr,
                                             qo_indptr, accept_len, accepted_nodes, batch, total_kv, max_depth, new_len,
                                             ddt::device_sm_count(), err, as_stream(stream)));
}

size_t ddt_cache_compact_workspace_size(int64_t pool_rows) {
    if (pool_rows < 1 || pool_rows > DDT_CACHE_MAX_ROWS) return 0;
    return ddt::cache_compact_workspace(pool_rows);
}

ddt_status ddt_cache_compact(void *slab, int64_t pool_bytes, int64_t pool_rows, int32_t num_pools,
                             int64_t row_bytes, const int32_t *kv_indices, int32_t total,
                             int32_t *new_indices, int32_t *live, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (bad_slab(slab, pool_bytes, pool_rows, num_pools, row_bytes) || total < 0 ||
        (total > 0 && (!kv_indices || !new_indices)) || !live)
        return DDT_ERR_INVALID_ARG;
    if (pool_rows > DDT_CACHE_MAX_ROWS) return DDT_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < ddt::cache_compact_workspace(pool_rows) || misaligned(workspace, 256))
        return DDT_ERR_WORKSPACE;
    // slots that are still read may not be written: in place each is, by its own reader
    if ((new_indices != kv_indices && overlap(new_indices, total, kv_indices, total)) ||
        overlap(live, 1, kv_indices, total) || overlap(live, 1, new_indices, total))
        return DDT_ERR_INVALID_ARG;
    unsigned int *err = ddt::device_error_word();
    if (!err) return DDT_ERR_CUDA;
    return launched(ddt::launch_cache_compact(slab, pool_bytes, pool_rows, num_pools, row_bytes, kv_indices, total,
                                              new_indices, live, workspace, ddt::device_sm_count(), err,
                                              as_stream(stream)));
}

ddt_status ddt_call_words(const int64_t *words) {
    if (!words) return DDT_ERR_INVALID_ARG;
    switch (words[0]) {
        case DDT_CALL_GQA_NORM_ROPE_APPEND: return call_words(ddt_gqa_norm_rope_append, words);
        case DDT_CALL_GQA_VERIFY_ATTN: return call_words(ddt_gqa_verify_attn, words);
        case DDT_CALL_CACHE_COPY: return call_words(ddt_cache_copy, words);
        case DDT_CALL_CACHE_COMMIT: return call_words(ddt_cache_commit, words);
        case DDT_CALL_CACHE_COMPACT: return call_words(ddt_cache_compact, words);
    }
    return DDT_ERR_INVALID_ARG;
}

}  // extern "C"
