// ddt_evict.cu -- a cache cut down to the columns that received most.
//
// Request b keeps min(N_b, budget_b) of its columns: in the order of their keys (the
// first `sinks` and the last `recent` columns and +inf on top, NaN with -inf at the
// bottom), ties to the lower column.  What stays keeps its order.
//
// A request has a cluster of CTAs, each with an equal run of its columns, whose weights it
// reads once and keeps as ordered 32-bit keys in shared memory.  The smallest key that stays is
// found by its bytes, highest first: a histogram of the keys that agree so far, summed over
// the cluster through distributed shared memory, and the byte at which the count reaches what
// is to stay.  Columns above that key stay, and of those with the key as many of the first
// ones as are left.  A count of both per warp, scanned over the CTA and the cluster, then gives
// every column its place.  Nothing depends on the order of atomics (they count).
//
// Bound by latency: a launch, one pass over 8 bytes a column, four histograms with a cluster
// barrier each, one pass that writes.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ddt_internal.cuh"
#include "ddt_sm100.cuh"

namespace ddt {
namespace {

using namespace sm100;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCopies = 4;           // of a histogram, against conflicts
constexpr int kMostKeys = 45056;     // of a CTA in shared memory; further ones are read again
constexpr int kColumnsOfCta = 8192;  // a cluster grows up to 16 CTAs to keep a CTA's columns below
constexpr uint32_t kTop = 0xff800000u;  // key of +inf
constexpr uint32_t kAll = 0xffffffffu;

struct EvictParams {
    EvictArgs a;
    int cluster;  // CTAs of a request
    int keys;     // of a CTA, in shared memory
};

// Floats as integers of the same order: -0 is 0, NaN is -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x != x ? -INFINITY : x);
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint32_t remote_u32(uint32_t local, uint32_t cta) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(local, cta)) : "memory");
    return v;
}
// columns of request b, or -1 where its offsets are broken
__device__ __forceinline__ int columns_of(const EvictArgs &a, int b) {
    const int kv0 = a.kv_indptr[b], kv1 = a.kv_indptr[b + 1];
    const int n = (int)((uint32_t)kv1 - (uint32_t)kv0);
    return kv0 < 0 || kv1 < kv0 || kv1 > a.total_kv || n > a.max_kv_len ? -1 : n;
}

__global__ void __launch_bounds__(kThreads, 1) evict_kernel(const __grid_constant__ EvictParams prm) {
    const EvictArgs &a = prm.a;
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t copies[256 * kCopies], counts[4][256], sums[256];
    __shared__ uint32_t above[kWarps], equal[kWarps], totals[2], found[2];
    __shared__ int64_t kept_before[kWarps], gone_before[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = prm.cluster, b = blockIdx.x / cluster, rank = blockIdx.x - b * cluster;
    auto sync_all = [&]() {  // and what the cluster's CTAs wrote is seen
        if (cluster > 1) cluster_sync();
        else __syncthreads();
    };
    pdl_wait();
    pdl_trigger();

    // ---- the request, and what the ones before it keep ----
    const int checked = columns_of(a, b), N = max(checked, 0);
    if (checked < 0 && rank == 0 && tid == 0) latch(a.err, DDT_DEVERR_KV_INDPTR);
    const int kept = min(N, max(a.budget[b], 0)), kv0 = a.kv_indptr[b];
    int64_t stay = 0, go = 0;
    for (int i = tid; i < b; i += kThreads) {
        const int n = max(columns_of(a, i), 0), k = min(n, max(a.budget[i], 0));
        stay += k;
        go += n - k;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        stay += __shfl_xor_sync(kAll, stay, o);
        go += __shfl_xor_sync(kAll, go, o);
    }
    if (lane == 0) {
        kept_before[warp] = stay;
        gone_before[warp] = go;
    }

    // ---- keys ----
    const int per = (int)((((int64_t)N + cluster - 1) / cluster + 31) & ~31);
    const int c0 = (int)min((int64_t)N, (int64_t)rank * per), n = min(per, N - c0);  // the CTA's columns
    const float *w = a.weights + kv0 + c0;
    const int recent_from = N - min(a.recent, N);
    auto make_key = [&](int i) {
        const int j = c0 + i;
        return j < a.sinks || j >= recent_from ? kTop : key_of(w[i]);
    };
    auto key = [&](int i) { return i < prm.keys ? keys[i] : make_key(i); };
    for (int i = tid; i < min(n, prm.keys); i += kThreads) keys[i] = make_key(i);
    for (int i = tid; i < 256 * kCopies; i += kThreads) copies[i] = 0;
    __syncthreads();

    // ---- the smallest key that stays, and how many columns that have it do ----
    uint32_t prefix = 0, mask = 0, left = kept;
    if (kept == N || kept == 0) {
        prefix = kept ? 0u : kAll;  // below and above every key
        left = 0;
    } else {
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            for (int i = tid; i < n; i += kThreads) {
                const uint32_t k = key(i);
                if ((k & mask) == prefix) atomicAdd(&copies[((k >> shift) & 255u) * kCopies + (lane & (kCopies - 1))], 1u);
            }
            __syncthreads();
            if (tid < 256) {
                uint32_t s = 0;
#pragma unroll
                for (int c = 0; c < kCopies; ++c) {
                    s += copies[tid * kCopies + c];
                    copies[tid * kCopies + c] = 0;
                }
                counts[pass][tid] = s;
            }
            sync_all();
            if (tid < 256) {
                uint32_t s = counts[pass][tid];
                if (cluster > 1) {
                    s = 0;
                    for (int r = 0; r < cluster; ++r) s += remote_u32(smem_u32(&counts[pass][tid]), r);
                }
                sums[tid] = s;
            }
            __syncthreads();
            if (warp == 0) {  // lane l has the bytes 255 - 8 l and the 7 below
                uint32_t v[8], mine = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = sums[255 - 8 * lane - i];
                    mine += v[i];
                }
                uint32_t upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_up_sync(kAll, upto, o);
                    if (lane >= o) upto += x;
                }
                const int at = __ffs(__ballot_sync(kAll, upto >= left)) - 1;
                if (lane == at) {
                    uint32_t before = upto - mine;
                    int i = 0;
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (i == e && before + v[e] < left) {
                            before += v[e];
                            i = e + 1;
                        }
                    found[0] = 255 - 8 * lane - i;
                    found[1] = left - before;
                }
            }
            __syncthreads();
            prefix |= found[0] << shift;
            mask |= 255u << shift;
            left = found[1];
        }
    }

    // ---- places ----
    // a warp has a run of the CTA's columns, which it goes through in order
    const int run = ((n + kWarps - 1) / kWarps + 31) & ~31, r0 = min(n, warp * run), r1 = min(n, r0 + run);
    uint32_t up = 0, same = 0;
    for (int i0 = r0; i0 < r1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < r1 ? key(i) : 0u;
        up += __popc(__ballot_sync(kAll, i < r1 && k > prefix));
        same += __popc(__ballot_sync(kAll, i < r1 && k == prefix));
    }
    if (lane == 0) {
        above[warp] = up;
        equal[warp] = same;
    }
    __syncthreads();
    if (warp == 0) {
        uint32_t u = above[lane], s = equal[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(kAll, u, o), y = __shfl_up_sync(kAll, s, o);
            if (lane >= o) {
                u += x;
                s += y;
            }
        }
        if (lane == 31) {
            totals[0] = u;
            totals[1] = s;
        }
        above[lane] = u - above[lane];
        equal[lane] = s - equal[lane];
    }
    sync_all();
    uint32_t up_before = above[warp], same_before = equal[warp];
    if (cluster > 1) {
        const uint32_t u = lane < rank ? remote_u32(smem_u32(&totals[0]), lane) : 0u;
        const uint32_t s = lane < rank ? remote_u32(smem_u32(&totals[1]), lane) : 0u;
        up_before += __reduce_add_sync(kAll, u);
        same_before += __reduce_add_sync(kAll, s);
        cluster_sync();  // no CTA leaves while another one reads its counts
    }
    int64_t base = 0, gone = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        base += kept_before[i];
        gone += gone_before[i];
    }
    if (rank == 0 && tid == 0) {
        if (b == 0) a.new_indptr[0] = 0;
        a.new_indptr[b + 1] = (int)(base + kept);
        if (base + kept > a.total_new || (a.evicted && gone + N - kept > a.total_evicted)) latch(a.err, DDT_DEVERR_KV_INDPTR);
    }
    for (int i0 = r0; i0 < r1; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < r1;
        const uint32_t k = in ? key(i) : 0u, lanes = (1u << lane) - 1u;
        const uint32_t ups = __ballot_sync(kAll, in && k > prefix), sames = __ballot_sync(kAll, in && k == prefix);
        const uint32_t u = up_before + __popc(ups & lanes), s = same_before + __popc(sames & lanes);
        if (in) {
            const bool stays = k > prefix || (k == prefix && s < left);
            const uint32_t stayed = u + min(s, left);  // of the request's columns before this one
            const int slot = a.kv_indices[kv0 + c0 + i];
            if (stays) {
                const int64_t to = base + stayed;
                if (to < a.total_new) {
                    a.new_indices[to] = slot;
                    if (a.new_weights) a.new_weights[to] = w[i];
                }
            } else if (a.evicted) {
                const int64_t to = gone + c0 + i - stayed;
                if (to < a.total_evicted) a.evicted[to] = slot;
            }
        }
        up_before += __popc(ups);
        same_before += __popc(sames);
    }
}

int cluster_of(int max_kv_len) {
    int c = 1;
    while (c < 16 && (int64_t)c * kColumnsOfCta < max_kv_len) c *= 2;
    return c;
}

}  // namespace

cudaError_t evict_prepare_device() {
    cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

cudaError_t launch_cache_evict(const EvictArgs &a, cudaStream_t s) {
    EvictParams prm;
    prm.a = a;
    prm.cluster = cluster_of(a.max_kv_len);
    const int64_t per = (((int64_t)a.max_kv_len + prm.cluster - 1) / prm.cluster + 31) & ~31;
    prm.keys = (int)std::min<int64_t>(per, kMostKeys);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(prm.cluster * a.batch));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)prm.keys * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)prm.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = prm.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel, prm);
}

}  // namespace ddt
