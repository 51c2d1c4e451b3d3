// ddt_gqa_chunk.cu -- chunk attention and received weights: sizes, the choice of how the work is split, launches.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "ddt_gqa_chunk_attn.cuh"
#include "ddt_gqa_chunk_weights.cuh"

namespace ddt {
namespace chunk {
extern template cudaError_t launch_attn_score<0>(AttnParams &, cudaStream_t);
extern template cudaError_t launch_attn_score<kCap>(AttnParams &, cudaStream_t);
extern template cudaError_t launch_attn_score<kBias>(AttnParams &, cudaStream_t);
extern template cudaError_t launch_attn_score<kCap | kBias>(AttnParams &, cudaStream_t);
extern template cudaError_t prepare_attn_score<0>();
extern template cudaError_t prepare_attn_score<kCap>();
extern template cudaError_t prepare_attn_score<kBias>();
extern template cudaError_t prepare_attn_score<kCap | kBias>();
namespace received {
extern template cudaError_t launch_weights_score<0>(Params &, int, cudaStream_t);
extern template cudaError_t launch_weights_score<kCap>(Params &, int, cudaStream_t);
extern template cudaError_t launch_weights_score<kBias>(Params &, int, cudaStream_t);
extern template cudaError_t launch_weights_score<kCap | kBias>(Params &, int, cudaStream_t);
extern template cudaError_t prepare_weights_score<0>();
extern template cudaError_t prepare_weights_score<kCap>();
extern template cudaError_t prepare_weights_score<kBias>();
extern template cudaError_t prepare_weights_score<kCap | kBias>();
}  // namespace received

namespace {
int part_rows(int tiles, int max_q_len, int group) { return (int)std::min<int64_t>((int64_t)max_q_len * group, tiles * kRows); }
int items_most(int tiles, int max_q_len, int group) {
    return (int)(((int64_t)max_q_len * group + tiles * kRows - 1) / (tiles * kRows));
}
bool may_deal(int batch, int max_kv_len) { return batch <= kChunkMaxDealtBatch && max_kv_len > 256; }
int slots(int tiles, int num_sms) { return std::min(num_sms * (tiles == 2 ? 1 : 2), DDT_GQA_MAX_CTAS); }
}  // namespace
}  // namespace chunk

using namespace chunk;

cudaError_t chunk_prepare_device() {
    cudaError_t e = prepare_attn_score<0>();
    if (e == cudaSuccess) e = prepare_attn_score<kCap>();
    if (e == cudaSuccess) e = prepare_attn_score<kBias>();
    if (e == cudaSuccess) e = prepare_attn_score<kCap | kBias>();
    if (e == cudaSuccess) e = received::prepare_weights_score<0>();
    if (e == cudaSuccess) e = received::prepare_weights_score<kCap>();
    if (e == cudaSuccess) e = received::prepare_weights_score<kBias>();
    if (e == cudaSuccess) e = received::prepare_weights_score<kCap | kBias>();
    return e;
}

int chunk_tiles(int max_q_len, int group) { return (int64_t)max_q_len * group > kRows ? 2 : 1; }

size_t chunk_layout(ChunkArgs &a, void *base) {
    const int group = a.num_heads / a.num_kv_heads;
    const size_t rows = (size_t)2 * a.num_ctas * part_rows(a.tiles, a.max_q_len, group);
    auto align = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t notes = align((size_t)a.num_ctas * sizeof(int4)), o = align(rows * a.head_dim * sizeof(float));
    if (base) {
        char *p = static_cast<char *>(base);
        a.notes = reinterpret_cast<int4 *>(p);
        a.o_part = reinterpret_cast<float *>(p + notes);
        a.lse_part = reinterpret_cast<float *>(p + notes + o);
    }
    return notes + o + align(rows * sizeof(float));
}

int chunk_most_ctas(int batch, int num_heads, int num_kv_heads, int max_q_len, int max_kv_len, int num_sms) {
    return may_deal(batch, max_kv_len) ? slots(chunk_tiles(max_q_len, num_heads / num_kv_heads), num_sms) : 0;
}

namespace {
// Microseconds that a call takes, roughly: with its blocks dealt to `ctas` CTAs, or (ctas = 0) with a CTA
// per item, which the hardware hands out as others end.  Dealing costs the plan, cut items and the join, and
// evens out long or few items; two tiles halve the reads of K and V, one tile starts and ends faster.  The
// constants are fitted to 104 shapes measured all four ways (plain scores alone; D = 128 with 64 heads on 8 and D =
// 64 with 16 heads, 17 to 1024 tokens, after 300 to 16000, 1 to 16 requests): each way within 24%, 5% on
// average.  The choice costs 1% over the best of the four on average and 20% at most; two tiles, dealt, cost
// 35% and 115%.  One chunk of 32 after 300 takes 27 us dealt with two tiles, 13 us with a CTA per item and one;
// 16 of 64 after 16000 433 us and 542 us; 16 of 32 after 4000 93 us dealt with two tiles, 73 us with a CTA per
// item.  The sizes are means over the call, and caps, slopes and a prefix that all tokens see are not known here.
double estimate(const ChunkArgs &a, int tiles, int ctas, int num_sms) {
    const double group = (double)a.num_heads / a.num_kv_heads, q = std::min((double)a.total_q / a.batch, (double)a.max_q_len);
    const double rows = q * group, items = (double)a.batch * a.num_kv_heads * std::ceil(rows / (tiles * kRows));
    const double window = a.window > 0 ? a.window + tiles * kRows / group : 1e30, block = 64.0 * tiles;
    const double mean = std::min(std::min((double)a.total_kv / a.batch, (double)a.max_kv_len) - q / 2, window) / block;
    const double most = std::min((double)a.max_kv_len, window) / block, w = a.head_dim / 128.0;
    if (ctas > 0) {
        const double all = rows * a.batch * a.num_kv_heads / 1000;
        return tiles == 1 ? 20.2 + items * (12.9 + 1.29 * (0.4 + 0.6 * w) * mean) / ctas + 0.014 * all
                          : 23.8 + items * 1.91 * (0.57 + 0.43 * w) * mean / ctas + 0.25 * all;
    }
    // one tile: two CTAs on an SM slow each other down
    const double per = tiles == 1 ? 0.9 * (0.72 + 0.28 * w) * (1 + 0.25 * std::min(std::max(items / num_sms - 1, 0.0), 1.0))
                                  : 1.7 * (0.73 + 0.27 * w);
    const double start = tiles == 1 ? 8.6 : 13.1, waves = items / (num_sms * (tiles == 1 ? 2 : 1));
    const double longest = start + per * most;  // the last CTAs to end may be of this kind
    return waves <= 1 ? longest : std::max(longest, waves * (start + per * mean) + 0.33 * longest);
}
}  // namespace

void chunk_choose(ChunkArgs &a, size_t workspace_bytes, int num_sms) {
    const int most_tiles = chunk_tiles(a.max_q_len, a.num_heads / a.num_kv_heads);
    int best_tiles = 1, best_ctas = 0;
    double best = 0;
    for (int tiles = 1; tiles <= most_tiles; ++tiles) {
        a.tiles = tiles;
        a.num_ctas = may_deal(a.batch, a.max_kv_len) ? slots(tiles, num_sms) : 0;
        while (a.num_ctas > 0 && chunk_layout(a, nullptr) > workspace_bytes) --a.num_ctas;
        for (int dealt = a.num_ctas > 0; dealt >= 0; --dealt) {
            const int ctas = dealt ? a.num_ctas : 0;
            const double us = estimate(a, tiles, ctas, num_sms);
            if (best == 0 || us < best) {
                best = us;
                best_tiles = tiles;
                best_ctas = ctas;
            }
        }
    }
    a.tiles = best_tiles;
    a.num_ctas = best_ctas;
}

namespace {
// cuTensorMapEncodeTiled from the driver, looked up once through the runtime
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}
// a pool with boxes of 16 rows x 64 values
bool encode_pool(CUtensorMap *map, const uint16_t *pool, const ChunkArgs &a) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)a.num_kv_heads * a.head_dim, (cuuint64_t)a.pool_rows};
    const cuuint64_t strides[1] = {(cuuint64_t)a.pool_stride * 2};
    const cuuint32_t box[2] = {64, 16}, elem[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(pool), dims, strides, box, elem,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

cudaError_t launch_chunk_attn(const ChunkArgs &a, int num_sms, cudaStream_t s) {
    AttnParams prm;
    memset(&prm, 0, sizeof prm);
    prm.a = a;
    if (!encode_pool(&prm.k_map, a.k_pool, a) || !encode_pool(&prm.v_map, a.v_pool, a)) return cudaErrorInvalidValue;
    prm.group = a.num_heads / a.num_kv_heads;
    prm.group_inv = 1.0f / (float)prm.group;
    prm.part_rows = part_rows(a.tiles, a.max_q_len, prm.group);
    prm.tgs_most = items_most(a.tiles, a.max_q_len, prm.group);
    prm.score = score_scale(a.scale, a.score_cap);
    prm.cap_most = a.score_cap / a.scale;
    switch ((a.score_cap > 0.f ? kCap : 0) | (a.slopes ? kBias : 0)) {
        case kCap: return launch_attn_score<kCap>(prm, s);
        case kBias: return launch_attn_score<kBias>(prm, s);
        case kCap | kBias: return launch_attn_score<kCap | kBias>(prm, s);
    }
    return launch_attn_score<0>(prm, s);
}

int chunk_weights_most_ctas(int batch, int num_sms) {
    return batch <= kChunkMaxDealtBatch ? std::min(num_sms, DDT_GQA_MAX_CTAS) : 0;
}

size_t chunk_weights_layout(ChunkArgs &a, void *base) {
    const size_t notes = ((size_t)a.num_ctas * sizeof(int4) + 255) & ~size_t(255);
    if (base) {
        a.notes = static_cast<int4 *>(base);
        a.o_part = reinterpret_cast<float *>(static_cast<char *>(base) + notes);
    }
    return notes + (size_t)2 * a.num_ctas * received::kCols * sizeof(float);
}

cudaError_t launch_chunk_weights(const ChunkArgs &a, const WeightArgs &w, cudaStream_t s) {
    received::Params prm;
    memset(&prm, 0, sizeof prm);
    prm.a = a;
    prm.w = w;
    prm.group = a.num_heads / a.num_kv_heads;
    prm.group_inv = 1.0f / (float)prm.group;
    prm.items_most = (int)(((int64_t)a.max_kv_len + received::kCols - 1) / received::kCols);
    prm.score = score_scale(a.scale, a.score_cap);
    prm.cap_most = a.score_cap / a.scale;
    const double log2e = a.score_cap > 0.f ? (double)prm.score.cap2 / a.score_cap : (double)prm.score.lin / a.scale;
    prm.log2e = (float)log2e;
    prm.log2e_rest = (float)(log2e - prm.log2e);
    const int rows = w.last_rows > 0 ? std::min(w.last_rows, a.max_q_len) : a.max_q_len;
    const int nq = (int64_t)rows * prm.group <= 16 ? 16 : 128;
    switch ((a.score_cap > 0.f ? kCap : 0) | (a.slopes ? kBias : 0)) {
        case kCap: return received::launch_weights_score<kCap>(prm, nq, s);
        case kBias: return received::launch_weights_score<kBias>(prm, nq, s);
        case kCap | kBias: return received::launch_weights_score<kCap | kBias>(prm, nq, s);
    }
    return received::launch_weights_score<0>(prm, nq, s);
}

}  // namespace ddt
