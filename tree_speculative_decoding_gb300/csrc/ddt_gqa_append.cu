// ddt_gqa_append.cu -- norm, rotation and cache append of a grouped-query
// layer's q, k and v in one pass.
//
// Per head row x of head_dim values: y = x * rsqrt(mean(x^2) + eps) * w, then
// the pairs of the first rope_dim values of q and k turned by the angle of the
// token's position, prefix + depth (the tree's root sits right behind the
// prefix, node n at its depth below it: "The Architecture of a Speculative
// Decoding Engine", section "The Final Resolution: A Concrete Trace").
//
// Bound by memory: 2 bytes in and 2 out per value, some twenty fp32 operations.
// A group of head_dim / 8 lanes holds one head row, 16 bytes a lane; the sum of
// squares and the far half of a pair come by shuffles inside the group, so the
// row is read once and written once.  One CTA takes a token (its request, slot
// and angles are looked up once) and its groups walk the token's q, k and v
// rows four at a time, loads first.  With few tokens several CTAs share one.
// The angles are read from the caller's table: sine and cosine of far
// positions need more than fp32, once per position and not per token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ddt_gqa.cuh"
#include "ddt_internal.cuh"

namespace ddt {
namespace {

constexpr int kThreads = 256;
constexpr int kBatchRows = 4;  // head rows in flight per group

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) norm_rope_append_kernel(const AppendArgs a) {
    constexpr int kLanes = D / 8;               // lanes of one head row
    constexpr int kGroups = kThreads / kLanes;  // head rows of a CTA at a time
    const int lane = threadIdx.x & 31;
    const int sub = threadIdx.x & (kLanes - 1);  // this lane's 8 values: [8 sub, 8 sub + 8)
    const int t = blockIdx.x;
    pdl_wait();
    pdl_trigger();  // after the wait: whatever runs next sees everything before this kernel

    const int b = find_request(a.qo_indptr, a.batch, t, lane);
    if (b >= a.batch) return;  // behind the last request: left as it is
    const int q0 = a.qo_indptr[b], T = a.qo_indptr[b + 1] - q0;
    const int kv0 = a.kv_indptr[b], kv1 = a.kv_indptr[b + 1];
    const int P = kv1 - kv0 - T;
    const bool bad_q = q0 < 0 || t - q0 >= T || q0 + T > a.total_q;
    const bool bad_kv = kv0 < 0 || kv1 > a.total_kv || P < 0;
    if (bad_q || bad_kv) {
        if (threadIdx.x == 0) latch(a.err, bad_q ? DDT_DEVERR_QO_INDPTR : DDT_DEVERR_KV_INDPTR);
        return;
    }
    const int i = t - q0;
    const int64_t slot = a.kv_indices[kv0 + P + i];
    const bool slot_ok = slot >= 0 && slot < a.pool_rows;
    if (!slot_ok && threadIdx.x == 0) latch(a.err, DDT_DEVERR_KV_INDEX);
    // this lane's angles: first half of a split pair, second half, or (interleaved) four whole pairs
    const int half = a.rope_dim >> 4;  // lanes of half the rotated values
    const bool turn = sub < 2 * half;
    float cs[8], sn[8];
    if (a.rope_dim > 0) {
        const int64_t pos = (int64_t)P + (a.depth ? a.depth[t] : i);
        if (pos < 0 || pos >= a.max_pos) {
            if (threadIdx.x == 0) latch(a.err, DDT_DEVERR_POSITION);
            return;
        }
        const float *row = a.cos_sin + pos * a.rope_dim;
        if (turn) {
            const int first = a.interleaved ? 4 * sub : 8 * (sub < half ? sub : sub - half);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (v == 1 && a.interleaved) break;
                const float4 c = *reinterpret_cast<const float4 *>(row + first + 4 * v);
                const float4 s = *reinterpret_cast<const float4 *>(row + (a.rope_dim >> 1) + first + 4 * v);
                cs[4 * v] = c.x; cs[4 * v + 1] = c.y; cs[4 * v + 2] = c.z; cs[4 * v + 3] = c.w;
                sn[4 * v] = s.x; sn[4 * v + 1] = s.y; sn[4 * v + 2] = s.z; sn[4 * v + 3] = s.w;
            }
        }
    }
    float wq[8], wk[8];
    if (a.q_weight) unpack8(reinterpret_cast<const uint4 *>(a.q_weight)[sub], wq);
    if (a.k_weight) unpack8(reinterpret_cast<const uint4 *>(a.k_weight)[sub], wk);

    const int H = a.num_heads, G = a.num_kv_heads;
    const int rows = H + 2 * G;
    const int group = blockIdx.y * kGroups + threadIdx.x / kLanes;
    const int stride = gridDim.y * kGroups;
    // lanes of a warp walk the same number of batches: the shuffles below need them all
    for (int base = group; __any_sync(0xffffffffu, base < rows); base += kBatchRows * stride) {
        uint4 in[kBatchRows];
#pragma unroll
        for (int u = 0; u < kBatchRows; ++u) {
            const int r = base + u * stride;
            const uint16_t *src = r < H ? a.q + t * a.q_stride + (int64_t)r * D
                : r < H + G ? a.k + t * a.k_stride + (int64_t)(r - H) * D
                            : a.v + t * a.v_stride + (int64_t)(r - H - G) * D;
            if (r < rows) in[u] = reinterpret_cast<const uint4 *>(src)[sub];
        }
#pragma unroll
        for (int u = 0; u < kBatchRows; ++u) {
            const int r = base + u * stride;
            if (!__any_sync(0xffffffffu, r < rows)) break;
            const bool is_q = r < H, is_v = r >= H + G;
            float x[8];
            unpack8(r < rows ? in[u] : make_uint4(0, 0, 0, 0), x);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, kLanes);
            if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr) {
                const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= inv * (is_q ? wq[e] : wk[e]);
            }
            if (a.rope_dim > 0) {
                if (a.interleaved) {
                    if (turn) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const float lo = x[2 * p], hi = x[2 * p + 1];
                            x[2 * p] = lo * cs[p] - hi * sn[p];
                            x[2 * p + 1] = hi * cs[p] + lo * sn[p];
                        }
                    }
                } else {
                    const int other = !turn ? sub : sub < half ? sub + half : sub - half;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = __shfl_sync(0xffffffffu, x[e], other, kLanes);
                        if (turn) x[e] = sub < half ? x[e] * cs[e] - y * sn[e] : x[e] * cs[e] + y * sn[e];
                    }
                }
            }
            if (r < rows && (is_q || slot_ok)) {
                uint16_t *dst = is_q ? a.q_out + ((int64_t)t * H + r) * D
                    : (is_v ? a.v_pool + (int64_t)(r - H - G) * D : a.k_pool + (int64_t)(r - H) * D) + slot * a.pool_stride;
                reinterpret_cast<uint4 *>(dst)[sub] = is_v ? in[u] : pack8(x);
            }
        }
    }
}

}  // namespace

cudaError_t launch_norm_rope_append(const AppendArgs &a, int num_sms, cudaStream_t s) {
    const int groups = kThreads / (a.head_dim / 8);
    const int rows = a.num_heads + 2 * a.num_kv_heads;
    // CTAs per token: one when the tokens alone fill the SMs, else down to one head row per group
    int split = (rows + groups - 1) / groups;
    const int64_t room = (4LL * num_sms + a.total_q - 1) / a.total_q;
    if (split > room) split = (int)room;
    const dim3 grid((unsigned)a.total_q, (unsigned)split);
    return a.head_dim == 128 ? launch_pdl(norm_rope_append_kernel<128>, grid, dim3(kThreads), 0, s, a)
                             : launch_pdl(norm_rope_append_kernel<64>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace ddt
