// ddt_gqa_attn.cu -- tree-verify attention over grouped-query K/V rows.
//
// One warp per (token, head): online softmax over the visible columns, fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ddt_internal.cuh"

namespace ddt {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int D>
__global__ void __launch_bounds__(128) gqa_attn_simple_kernel(const GqaArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.x * 4 + (threadIdx.x >> 5);
    const int i = blockIdx.y, b = blockIdx.z;
    pdl_wait();
    pdl_trigger();
    if (h >= a.num_heads) return;
    const int qo0 = a.qo_indptr[b], T = a.qo_indptr[b + 1] - qo0;
    const int kv0 = a.kv_indptr[b], kv1 = a.kv_indptr[b + 1], N = kv1 - kv0;
    const int m0 = a.mask_indptr[b], m1 = a.mask_indptr[b + 1], W = (N + 31) >> 5;
    const bool bad_qo = T < 0 || T > a.max_q_len || qo0 < 0 || qo0 + T > a.total_q;
    const bool bad_kv = N < T || N > a.max_kv_len || kv0 < 0 || kv1 > a.total_kv;
    const bool bad_mask = !bad_qo && !bad_kv && (m0 < 0 || m1 - m0 != T * W || m1 > a.total_mask_words);
    if (bad_qo || bad_kv || bad_mask) {
        if (lane == 0)
            latch(a.err, (bad_qo ? DDT_DEVERR_QO_INDPTR : 0u) | (bad_kv ? DDT_DEVERR_KV_INDPTR : 0u) |
                             (bad_mask ? DDT_DEVERR_MASK_INDPTR : 0u));
        return;
    }
    if (i >= T) return;
    const int g = h / (a.num_heads / a.num_kv_heads);
    const int64_t row = (int64_t)(qo0 + i) * a.num_heads + h;
    float q[E], o[E];
    for (int e = 0; e < E; ++e) {
        q[e] = __uint_as_float((uint32_t)a.q[row * D + lane * E + e] << 16);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const uint32_t *words = a.mask + m0 + (int64_t)i * W;
    for (int j = 0; j < N; ++j) {
        if (!((words[j >> 5] >> (j & 31)) & 1u)) continue;
        int64_t slot = a.kv_indices[kv0 + j];
        if (slot < 0 || slot >= a.pool_rows) {
            if (lane == 0) latch(a.err, DDT_DEVERR_KV_INDEX);
            slot = 0;
        }
        const int64_t at = slot * a.pool_stride + (int64_t)g * D + lane * E;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s = fmaf(q[e], __uint_as_float((uint32_t)a.k_pool[at + e] << 16), s);
        for (int w = 16; w >= 1; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= a.scale * kLog2e;
        const float mn = fmaxf(m, s);
        const float c = mn == -INFINITY ? 1.f : exp2f(m - mn), p = mn == -INFINITY ? 0.f : exp2f(s - mn);
        m = mn;
        l = l * c + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * __uint_as_float((uint32_t)a.v_pool[at + e] << 16);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int e = 0; e < E; ++e) {
        const __nv_bfloat16 r = __float2bfloat16_rn(o[e] * inv);
        a.out[row * D + lane * E + e] = *reinterpret_cast<const uint16_t *>(&r);
    }
    if (a.lse && lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

int gqa_choose_splits(int, int, int, int, int, int, int) { return 1; }

void gqa_split_layout(int max_kv_len, int, int *split_cols, int *splits) {
    *split_cols = max_kv_len;
    *splits = 1;
}

cudaError_t launch_gqa_attn(const GqaArgs &a, cudaStream_t s) {
    const dim3 grid((unsigned)((a.num_heads + 3) / 4), (unsigned)a.max_q_len, (unsigned)a.batch);
    return a.head_dim == 128 ? launch_pdl(gqa_attn_simple_kernel<128>, grid, dim3(128), 0, s, a)
                             : launch_pdl(gqa_attn_simple_kernel<64>, grid, dim3(128), 0, s, a);
}

}  // namespace ddt
