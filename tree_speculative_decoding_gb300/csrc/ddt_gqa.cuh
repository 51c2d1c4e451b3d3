// ddt_gqa.cuh -- device code shared by the grouped-query kernels.
#pragma once

#include <stdint.h>

namespace ddt {

// The last request b in [0, batch] with qo_indptr[b] <= t, by a 32-way search
// of the whole warp (two rounds of loads up to 1024 requests).  b == batch:
// the token is behind the last request.  0 is also the answer for a token ahead of
// the first one, and offsets that fall somewhere may give a b with qo_indptr[b] > t.
__device__ __forceinline__ int find_request(const int32_t *qo_indptr, int batch, int t, int lane) {
    int64_t lo = 0, hi = batch;
    while (hi > lo) {
        const int64_t step = (hi - lo + 31) >> 5;
        const int64_t probe = lo + (lane + 1) * step;
        const bool below = probe <= hi && qo_indptr[probe] <= t;
        const int64_t c = __popc(__ballot_sync(0xffffffffu, below));
        lo += c * step;
        if (lo + step - 1 < hi) hi = lo + step - 1;
    }
    return (int)lo;
}

}  // namespace ddt
