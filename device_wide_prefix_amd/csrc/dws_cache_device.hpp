// Device pieces shared by the kernels on cached keys and values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dws_cache.h"

namespace dws {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// What a wave's lanes wrote to the LDS is there for its other lanes.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ int64_t seq_begin(const KvView& c, int64_t i)
{
    return c.offsets != nullptr ? c.offsets[i] : i * c.each;
}

// The sequence that holds token t, -1 if none does, and its first token and
// length. Every lane of the wave calls it with the same t; 64 candidates a round,
// since a round is one trip to memory. (A sequence that begins before row 0 holds
// none: with 0 <= first <= t < end no difference of the three leaves 64 bits.)
__device__ __forceinline__ int64_t seq_of(const KvView& c, int64_t t, int64_t* first, int64_t* count, int lane)
{
    if (c.n == 0) return -1;
    int64_t i;
    if (c.offsets == nullptr) {
        i = t / c.each;
    } else {
        int64_t lo = 0, hi = c.n - 1;
        while (hi > lo) {
            const int64_t step = (hi - lo) / 64 + 1, at = lo + lane * step;
            const uint64_t found = __ballot(at <= hi && c.offsets[at <= hi ? at : hi] <= t);
            lo += found == 0 ? 0 : (63 - __builtin_clzll(found)) * step;
            if (found == 0) hi = lo;
            if (lo + step - 1 < hi) hi = lo + step - 1;
        }
        i = lo;
    }
    const int64_t b = seq_begin(c, i), e = seq_begin(c, i + 1);
    if (b < 0 || b > t || e <= t) return -1;
    *first = b;
    *count = e - b;
    return i;
}

}  // namespace dws
