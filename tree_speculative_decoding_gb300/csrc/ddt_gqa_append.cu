// ddt_gqa_append.cu -- norm, rotation and cache append of a grouped-query
// layer's q, k and v in one pass.
//
// Per head row x of head_dim values: y = x * rsqrt(mean(x^2) + eps) * w, then
// the pairs of the first rope_dim values of q and k turned by the angle of the
// token's position, prefix + depth (the tree's root sits right behind the
// prefix, node n at its depth below it: "The Architecture of a Speculative
// Decoding Engine", section "The Final Resolution: A Concrete Trace").
//
// Bound by memory: 2 bytes in and 2 out per value, some ten fp32 instructions
// per pair of values.  A group of head_dim / 8 lanes holds one head row.  A lane
// holds both halves of its pairs (two pieces of four values, rope_dim / 2
// apart), so the rotation needs no exchange between lanes; only the sum of
// squares crosses the group.  Weight, cosine and sine are folded into four
// factors per pair once per token.  A CTA takes a token and its groups walk the
// token's rows.  What bounds a CTA is its chain of dependent loads, so the first
// rows, the weights and the depth are loaded before the token's request is looked
// up, and its slot and angles at once behind that.  4096 tokens of 64 query and 8
// K/V heads of 128 in 32 requests take 29.3 us, 5.8 TB/s (30.5 us with 64 threads and
// 14 CTAs per SM, 33.5 us with 128 and 8; 39.6 us with 24 of these, 30.5 us with 32).
// With few tokens several CTAs share one.  The angles are read from the caller's
// table: sine and cosine of far positions need more than fp32, once per position and
// not per token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ddt_gqa.cuh"
#include "ddt_internal.cuh"
#include "ddt_sm100.cuh"

namespace ddt {
namespace {

using namespace sm100;

constexpr int kThreads = 32;
constexpr int kCtasPerSm = 28;
constexpr int kBatchRows = 4;  // head rows in flight per group

struct Row {  // a lane's two pieces of four values
    uint2 a, b;
};
__device__ __forceinline__ Row load_row(const uint16_t *p, int off0, int off1) {
    Row r;
    r.a = *reinterpret_cast<const uint2 *>(p + off0);
    r.b = *reinterpret_cast<const uint2 *>(p + off1);
    return r;
}
__device__ __forceinline__ void store_row(uint16_t *p, int off0, int off1, const Row &r) {
    *reinterpret_cast<uint2 *>(p + off0) = r.a;
    *reinterpret_cast<uint2 *>(p + off1) = r.b;
}
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The factors of a token's rows: out_a = a * aa + b * ab, out_b = b * bb + a * ba
// for the values a, b of a pair, times the row's 1 / rms.  With split pairs the
// two pieces are the two sides; with adjacent pairs the sides alternate inside
// each piece, and (a, b) are the values of one float2.
struct Factors {
    float2 aa[2], ab[2], bb[2], ba[2];
};

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) norm_rope_append_kernel(const AppendArgs a) {
    constexpr int kLanes = D / 8;               // lanes of one head row
    constexpr int kGroups = kThreads / kLanes;  // head rows of a CTA at a time
    const int lane = threadIdx.x & 31;
    const int sub = threadIdx.x & (kLanes - 1);
    const int t = blockIdx.x;
    const int H = a.num_heads, G = a.num_kv_heads;
    const int group = blockIdx.y * kGroups + threadIdx.x / kLanes;
    const int stride = gridDim.y * kGroups;
    // the lane's pieces: a pair's two sides, or eight values in a row (adjacent pairs, or not rotated)
    const int half = a.rope_dim >> 1;
    const bool turn = 8 * sub < a.rope_dim, split = turn && !a.interleaved;
    const int off0 = split ? 4 * sub : 8 * sub, off1 = split ? half + 4 * sub : 8 * sub + 4;
    pdl_wait();
    pdl_trigger();  // after the wait: whatever runs next sees everything before this kernel

    const uint16_t *q = a.q + t * a.q_stride;
    Row in[kBatchRows];
    auto load_batch = [&](int r0) {
#pragma unroll
        for (int u = 0; u < kBatchRows; ++u)
            if (r0 + u * stride < H) in[u] = load_row(q + (int64_t)(r0 + u * stride) * D, off0, off1);
    };
    load_batch(group);
    Row w_q{}, w_k{};  // the weights of the lane's values
    if (a.q_weight) w_q = load_row(a.q_weight, off0, off1);
    if (a.k_weight) w_k = load_row(a.k_weight, off0, off1);
    const int depth = a.depth ? a.depth[t] : 0;

    // The token's request: up to 31 requests one round of loads gives every offset
    // there is, else the search comes first.
    int b, q0, q1, kv0, kv1;
    if (a.batch < 32) {
        const int i = min(lane, a.batch);
        const int qo = a.qo_indptr[i], kv = a.kv_indptr[i];
        b = __popc(__ballot_sync(0xffffffffu, lane >= 1 && lane <= a.batch && qo <= t));
        q0 = __shfl_sync(0xffffffffu, qo, b);
        q1 = __shfl_sync(0xffffffffu, qo, b + 1);
        kv0 = __shfl_sync(0xffffffffu, kv, b);
        kv1 = __shfl_sync(0xffffffffu, kv, b + 1);
        if (b >= a.batch || (b == 0 && t < q0)) return;  // behind the last request or ahead of the first: left as it is
    } else {
        b = find_request(a.qo_indptr, a.batch, t, lane);
        if (b >= a.batch) return;
        q0 = a.qo_indptr[b];
        if (b == 0 && t < q0) return;
        q1 = a.qo_indptr[b + 1];
        kv0 = a.kv_indptr[b];
        kv1 = a.kv_indptr[b + 1];
    }
    const int64_t T = (int64_t)q1 - q0, P = (int64_t)kv1 - kv0 - T;  // broken offsets do not fit 32 bits
    // t < q0: offsets that fall somewhere lead the look-up to a request that starts behind the token
    const bool bad_q = q0 < 0 || t < q0 || t - q0 >= T || q1 > a.total_q;
    const bool bad_kv = kv0 < 0 || kv1 > a.total_kv || P < 0;
    if (bad_q || bad_kv) {
        if (threadIdx.x == 0) latch(a.err, bad_q ? DDT_DEVERR_QO_INDPTR : DDT_DEVERR_KV_INDPTR);
        return;
    }
    const int i = t - q0;
    const int64_t slot = a.kv_indices[kv0 + P + i];
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};  // of the lane's four pairs
    if (a.rope_dim > 0) {
        const int64_t pos = P + (a.depth ? depth : i);
        if (pos < 0 || pos >= a.max_pos) {
            if (threadIdx.x == 0) latch(a.err, DDT_DEVERR_POSITION);
            return;
        }
        if (turn) {
            const float *row = a.cos_sin + pos * a.rope_dim + 4 * sub;
            const float4 c = *reinterpret_cast<const float4 *>(row), s = *reinterpret_cast<const float4 *>(row + half);
            cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
            sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
        }
    }
    const bool slot_ok = slot >= 0 && slot < a.pool_rows;
    if (!slot_ok && threadIdx.x == 0) latch(a.err, DDT_DEVERR_KV_INDEX);
    auto factors = [&](bool weighted, const Row &w) {
        float2 w0[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, w1[2] = {w0[0], w0[1]};
        if (weighted) {
            w0[0] = unpack2(w.a.x); w0[1] = unpack2(w.a.y);
            w1[0] = unpack2(w.b.x); w1[1] = unpack2(w.b.y);
        }
        Factors f;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (a.interleaved) {  // pairs 2 p' and 2 p' + 1 of piece p: (x, y) = (a, b)
                const float c0 = cs[2 * p], c1 = cs[2 * p + 1], s0 = sn[2 * p], s1 = sn[2 * p + 1];
                const float2 wa = p ? w1[0] : w0[0], wb = p ? w1[1] : w0[1];
                f.aa[p] = make_float2(wa.x * c0, wb.x * c1);
                f.ab[p] = make_float2(-wa.y * s0, -wb.y * s1);
                f.bb[p] = make_float2(wa.y * c0, wb.y * c1);
                f.ba[p] = make_float2(wa.x * s0, wb.x * s1);
            } else {
                const float2 c = make_float2(cs[2 * p], cs[2 * p + 1]), s = make_float2(sn[2 * p], sn[2 * p + 1]);
                f.aa[p] = make_float2(w0[p].x * c.x, w0[p].y * c.y);
                f.ab[p] = make_float2(-w1[p].x * s.x, -w1[p].y * s.y);
                f.bb[p] = make_float2(w1[p].x * c.x, w1[p].y * c.y);
                f.ba[p] = make_float2(w0[p].x * s.x, w0[p].y * s.y);
            }
        }
        return f;
    };
    // one row; the whole warp calls it (lanes without a row pass anything)
    auto apply = [&](const Row &r, const Factors &f, bool norm) {
        float2 x[2][2] = {{unpack2(r.a.x), unpack2(r.a.y)}, {unpack2(r.b.x), unpack2(r.b.y)}};
        float inv = 1.f;
        if (norm) {
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int e = 0; e < 2; ++e) ss = f2fma(x[p][e], x[p][e], ss);
            float s = ss.x + ss.y;
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o, kLanes);
            inv = rsqrtf(s * (1.0f / D) + a.eps);
        }
        const float2 z = make_float2(0.f, 0.f), iv = make_float2(inv, inv);
        Row y;
        if (a.interleaved) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {  // the piece's two pairs
                const float2 xa = make_float2(x[p][0].x, x[p][1].x), xb = make_float2(x[p][0].y, x[p][1].y);
                const float2 ya = f2fma(f2fma(xa, f.aa[p], turn ? f2fma(xb, f.ab[p], z) : z), iv, z);
                const float2 yb = f2fma(f2fma(xb, f.bb[p], turn ? f2fma(xa, f.ba[p], z) : z), iv, z);
                (p ? y.b : y.a) = make_uint2(pack_bf16(ya.x, yb.x), pack_bf16(ya.y, yb.y));
            }
        } else {
            uint32_t wa[2], wb[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const float2 ya = f2fma(f2fma(x[0][p], f.aa[p], turn ? f2fma(x[1][p], f.ab[p], z) : z), iv, z);
                const float2 yb = f2fma(f2fma(x[1][p], f.bb[p], turn ? f2fma(x[0][p], f.ba[p], z) : z), iv, z);
                wa[p] = pack_bf16(ya.x, ya.y);
                wb[p] = pack_bf16(yb.x, yb.y);
            }
            y.a = make_uint2(wa[0], wa[1]);
            y.b = make_uint2(wb[0], wb[1]);
        }
        return y;
    };

    uint16_t *q_out = a.q_out + (int64_t)t * H * D;
    {
        const Factors f = factors(a.q_weight != nullptr, w_q);
        // groups of a warp walk the same number of rows: the sums above need all its lanes
        for (int r0 = group; __any_sync(0xffffffffu, r0 < H); r0 += kBatchRows * stride) {
            if (r0 != group) load_batch(r0);
#pragma unroll
            for (int u = 0; u < kBatchRows; ++u) {
                const int r = r0 + u * stride;
                if (!__any_sync(0xffffffffu, r < H)) break;
                const Row y = apply(in[u], f, a.q_weight != nullptr);
                if (r < H) store_row(q_out + (int64_t)r * D, off0, off1, y);
            }
        }
    }
    if (!slot_ok) return;  // the whole CTA
    const Factors f = factors(a.k_weight != nullptr, w_k);
    const uint16_t *k = a.k + t * a.k_stride, *v = a.v + t * a.v_stride;
    uint16_t *kp = a.k_pool + slot * a.pool_stride, *vp = a.v_pool + slot * a.pool_stride;
    for (int r = group; __any_sync(0xffffffffu, r < G); r += stride) {
        Row kr{}, vr{};
        if (r < G) {
            kr = load_row(k + (int64_t)r * D, off0, off1);
            vr = load_row(v + (int64_t)r * D, off0, off1);
        }
        kr = apply(kr, f, a.k_weight != nullptr);
        if (r < G) {
            store_row(kp + (int64_t)r * D, off0, off1, kr);
            store_row(vp + (int64_t)r * D, off0, off1, vr);
        }
    }
}

}  // namespace

cudaError_t launch_norm_rope_append(const AppendArgs &a, int num_sms, cudaStream_t s) {
    const int groups = kThreads / (a.head_dim / 8);
    // CTAs per token: as many as run at once, down to two query rows per group, and one
    // when the tokens alone fill the SMs.  1056 tokens of 64 query and 8 K/V heads of
    // 128: four take 7.4 us, more than one wave 9.2 us, one 9.5 us; 128 tokens: 3.0 us
    // with sixteen, 4.6 us with thirty-two, 5.8 us with one.
    const int64_t room = (int64_t)kCtasPerSm * num_sms / a.total_q;
    const int split = (int)std::max<int64_t>(1, std::min<int64_t>((a.num_heads + 2 * groups - 1) / (2 * groups), room));
    const dim3 grid((unsigned)a.total_q, (unsigned)split);
    return a.head_dim == 128 ? launch_pdl(norm_rope_append_kernel<128>, grid, dim3(kThreads), 0, s, a)
                             : launch_pdl(norm_rope_append_kernel<64>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace ddt
