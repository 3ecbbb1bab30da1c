// extents.h -- counts and walks over sizes up to 2^31 - 1 without a wrap in 32 bits, for host
// and device.
#pragma once
#include <stdint.h>

#if defined(__HIP__)
#include <hip/hip_runtime.h>
#define DG_HD __host__ __device__ __forceinline__
#else
#define DG_HD inline
#endif

namespace dg {

// Pieces of `of` (a power of two) that cover n >= 0: n + of - 1 would wrap near 2^31.
template <int of>
DG_HD int pieces(int n) {
    static_assert((of & (of - 1)) == 0, "a power of two");
    return n / of + (n % of != 0 ? 1 : 0);
}

// a + b or, where that is more, cap.
DG_HD int capped_sum(int a, int b, int cap) {
    const int64_t sum = (int64_t)a + b;
    return sum < cap ? (int)sum : cap;
}

// Calls f(at) for at = first, first + step, .. below end: a 32-bit counter would wrap past an
// end within one step of 2^31.
template <typename F>
DG_HD void stride_walk(int64_t first, int64_t end, int64_t step, F f) {
    for (int64_t at = first; at < end; at += step) f((int)at);
}

}  // namespace dg
