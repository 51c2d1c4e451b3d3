// ddt_gqa_chunk.cuh -- what the chunk kernels share: which columns a token sees,
// how a score is made of a product, and the range of columns that a run of tokens reads.
//
// Token i of a request with P cached columns is at position p = P + i, column j at
// position j.  It sees column j when j < full (a prefix that every token sees) or
// p - window < j <= p (window 0: j <= p).  Its score is
//   z = scale <q, k_j>;  z = cap tanh(z / cap) where cap > 0;  z -= slope |p - j|.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ddt_internal.cuh"
#include "ddt_sm100.cuh"

namespace ddt {
namespace chunk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kCap = 1, kBias = 2;  // bits of a kernel's kScore

constexpr uint32_t kWaitLimit = 1u << 17;  // of 20 us

// Waits that give up.  A wait sleeps in the barrier for up to 20 us at a time: the short default makes
// the waiting warps poll, and their instructions took a tenth of the attention's time (a prompt of 8192
// 1068 us, with longer sleeps 914).  The abort flag is read only where the phase is still open.
__device__ __forceinline__ bool mbar_sleep_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000; "
        "selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *err) {
    if (mbar_sleep_wait(bar, parity)) return true;
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (mbar_sleep_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    *abort = 1;
    latch(err, DDT_DEVERR_TIMEOUT);
    return false;
}
// The same for a whole warp: it succeeds for every lane or for none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *err) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort, err));
}

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {  // a, b >= 0; nearly always small enough for 32 bits
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// CTA c has the positions [lo, hi) of the line: [c q + min(c, rem), ...).
struct Shares {
    int64_t q, rem;
    __device__ __forceinline__ int64_t lo(int64_t c) const { return c * q + (c < rem ? c : rem); }
    __device__ __forceinline__ int owner(int64_t x) const {  // the CTA whose share holds position x
        const int64_t cut = rem * (q + 1);
        return (int)(x < cut ? divide(x, q + 1) : rem + divide(x - cut, q));
    }
};

// A request's offsets, checked: T new tokens behind N - T cached columns.
struct Request {
    int qo0, T, kv0, N, full;
};
__device__ __forceinline__ Request load_request(const ChunkArgs &a, int b, unsigned int *err) {
    Request r;
    r.qo0 = a.qo_indptr[b];
    const int qo1 = a.qo_indptr[b + 1];
    r.kv0 = a.kv_indptr[b];
    const int kv1 = a.kv_indptr[b + 1];
    r.full = a.full_len ? a.full_len[b] : 0;
    // differences of broken offsets wrap, which is why their order counts
    r.T = (int)((uint32_t)qo1 - (uint32_t)r.qo0);
    r.N = (int)((uint32_t)kv1 - (uint32_t)r.kv0);
    const bool bad_qo = r.T < 0 || r.T > a.max_q_len || r.qo0 < 0 || qo1 > a.total_q || qo1 < r.qo0;
    const bool bad_kv = r.N < r.T || r.N > a.max_kv_len || r.kv0 < 0 || kv1 > a.total_kv || kv1 < r.kv0;
    if (bad_qo || bad_kv) {
        latch(err, (bad_qo ? DDT_DEVERR_QO_INDPTR : 0u) | (bad_kv ? DDT_DEVERR_KV_INDPTR : 0u));
        r.T = r.N = 0;
    }
    r.full = min(max(r.full, 0), r.N);
    return r;
}

// n / group for 0 <= n < 128 * 128, 1 <= group <= 128 by the reciprocal: (n + 1/2) /
// group is at least 1/256 from a whole number, and off by less than 16384.5 * 2^-22.
__device__ __forceinline__ int quotient(int n, float group_inv) { return (int)(((float)n + 0.5f) * group_inv); }

// Blocks of NB columns that tokens at positions [pa, pb] read: 0 .. a - 1 for the
// prefix that all see, l .. r - 1 for the rest.
struct Blocks {
    int a, l, count;
};
template <int NB>
__device__ __forceinline__ Blocks blocks_of(int pa, int pb, int window, int full) {
    Blocks x;
    const int lo = window > 0 ? max(0, pa - window + 1) : 0;
    x.a = (full + NB - 1) / NB;
    x.l = max(x.a, lo / NB);
    x.count = x.a + max(x.l, pb / NB + 1) - x.l;
    return x;
}

// whether tokens at positions [pa, pb] all see columns [c, c + n)
__device__ __forceinline__ bool all_see(int c, int n, int pa, int pb, int window, int full) {
    return c + n <= full || (c + n - 1 <= pa && (window <= 0 || c > pb - window));
}
// the low n bits (n may be negative or above 32)
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
// bit e: the token at position p sees column c + e (of N)
__device__ __forceinline__ uint32_t seen_bits(int c, int p, int window, int full, int N) {
    uint32_t w = low_bits(p + 1 - c);
    if (window > 0) w &= ~low_bits(p - window + 1 - c);
    return (w | low_bits(full - c)) & low_bits(N - c);
}

// 32 consecutive 32-bit columns of this thread's lane, and the largest of them (kAbs: the largest
// magnitude) as floats; NaN counts only where all are.
template <bool kAbs>
__device__ __forceinline__ void tmem_ld32_max(uint32_t taddr, uint32_t (&r)[32], float &most) {
#define DDT_LD32_MAX(abs)                                                                                                      \
    asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x32.max" abs ".f32 "                                                      \
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"                                                     \
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"                               \
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), \
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),      \
                   "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),     \
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(most)       \
                 : "r"(taddr))
    if constexpr (kAbs) DDT_LD32_MAX(".abs");
    else DDT_LD32_MAX("");
#undef DDT_LD32_MAX
}

// A pair of scores in log2 units less a reference, from the products of q with columns j
// and j + 1 (where kBias: at distances p - j = -d, -d - 1).  tanh(u) = 1 - 2 / (1 + e^2u):
// off by 2^-22 at most, which is cap 2^-22 in a score; it stays right where e^2u is 0 or infinite.
struct ScoreScale {
    float lin;    // plain: scale log2(e); capped: 2 log2(e) scale / cap
    float cap2;   // cap log2(e)
    float u;      // scale / cap
    float slope;  // of the row's head, log2 units
};
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int kScore>
__device__ __forceinline__ float2 score_pair(float s0, float s1, const ScoreScale &k, float add0, float add1) {
    using namespace sm100;
    if constexpr (kScore & kCap) {
        const float2 t = f2fma(make_float2(s0, s1), make_float2(k.lin, k.lin), make_float2(0.f, 0.f));
        const float2 w = f2add(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
        return f2fma(make_float2(rcp(w.x), rcp(w.y)), make_float2(-2.f * k.cap2, -2.f * k.cap2),
                     f2add(make_float2(add0, add1), make_float2(k.cap2, k.cap2)));
    } else {
        return f2fma(make_float2(s0, s1), make_float2(k.lin, k.lin), make_float2(add0, add1));
    }
}
// The same where every |z / cap| of the pair is below 1: cap tanh(u) = cap u P(u^2), P of degree 6 with the
// least largest error of u P(u^2) over [0, 1] (Lawson's weighted least squares, coefficients rounded one after
// another and the rest fitted again: 2.0e-8; in fp32 6.4e-8 at most, measured over the range).  Ten multiply-adds in place of two special functions, of which a reciprocal takes 8 cycles of
// a warp's share of the unit and 2^x 4.  The factors are pairs in registers: a packed multiply-add takes
// no immediate, and read from constant memory they took longer than the special functions.
struct CapPoly {
    uint64_t u, cap2, c[7];
    __device__ __forceinline__ static uint64_t both(float x) {
        uint64_t r;
        asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));  // (volatile: made once, not at every use)
        return r;
    }
    __device__ __forceinline__ void set(const ScoreScale &k) {
        constexpr float kP[7] = {0.99999970198f, -0.33332145214f, 0.13319680095f, -0.053268551826f, 0.01997718215f, -0.0059540499933f, 0.00096454482991f};
        u = both(k.u);
        cap2 = both(k.cap2);
#pragma unroll
        for (int i = 0; i < 7; ++i) c[i] = both(kP[i]);
    }
};
__device__ __forceinline__ float2 score_pair_poly(float s0, float s1, const CapPoly &k, float add0, float add1) {
    float2 x;
    asm("{ .reg .b64 u, t, y, z; mov.b64 u, {%2, %3}; mul.rn.f32x2 u, u, %6; mul.rn.f32x2 t, u, u; "
        "fma.rn.f32x2 y, %14, t, %13; fma.rn.f32x2 y, y, t, %12; fma.rn.f32x2 y, y, t, %11; fma.rn.f32x2 y, y, t, %10; "
        "fma.rn.f32x2 y, y, t, %9; fma.rn.f32x2 y, y, t, %8; mul.rn.f32x2 u, u, %7; mov.b64 z, {%4, %5}; "
        "fma.rn.f32x2 z, u, y, z; mov.b64 {%0, %1}, z; }"
        : "=f"(x.x), "=f"(x.y)
        : "f"(s0), "f"(s1), "f"(add0), "f"(add1), "l"(k.u), "l"(k.cap2), "l"(k.c[0]), "l"(k.c[1]), "l"(k.c[2]), "l"(k.c[3]),
          "l"(k.c[4]), "l"(k.c[5]), "l"(k.c[6]));
    return x;
}
// (in 64 bits, with one rounding each: an error here is one of every score, and does not average out)
inline ScoreScale score_scale(double scale, double cap) {
    constexpr double log2e = 1.4426950408889634;
    ScoreScale k;
    k.lin = (float)(cap > 0 ? 2 * log2e * scale / cap : scale * log2e);
    k.cap2 = (float)(cap * log2e);
    k.u = (float)(cap > 0 ? scale / cap : 0);
    k.slope = 0.f;
    return k;
}

}  // namespace chunk
}  // namespace ddt
