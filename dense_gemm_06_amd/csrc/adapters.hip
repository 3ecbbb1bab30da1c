// adapters.hip -- low-rank adapters of many requests beside a shared product, in fp32.
//
//   u[t] = scale a_i x[t]      (shrink)        out[t] = base[t] + scale b_i u[t]   (expand)
//   a_grad_i = sum_t v[t] x[t]^T over adapter i's rows                             (gradient)
//
// The same kernels serve the backward pass with the roles of a and b exchanged, which differ
// in the direction that lies along memory (`turned`). Bound by loads: every row and every adapter comes from
// the caches for each token or element again (512 tokens, 1024 x 1024, rank 12, 3 adapters with the shared
// products, both ways: 122 us, of which these kernels take 27).
#include "device_common.h"
#include "layers.h"
#include "launch.h"

namespace dg {

namespace {

__device__ __forceinline__ float element(const void* p, size_t i) { return static_cast<const float*>(p)[i]; }

__device__ __forceinline__ size_t m_at(const AdapterArgs& a, int i, int j, int64_t k) {
    return (size_t)i * (size_t)a.stride_m +
           (a.turned ? (size_t)k * (size_t)a.ldm + (size_t)j : (size_t)j * (size_t)a.ldm + (size_t)k);
}

}  // namespace

// One wave: one token and one of its rank numbers.
__global__ __launch_bounds__(256) void adapter_shrink(AdapterArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t units = (int64_t)a.tokens * a.rank;
    for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < units; unit += (int64_t)gridDim.x * 4) {
        const int t = (int)(unit / a.rank), j = (int)(unit - (int64_t)t * a.rank);
        const int i = a.index[t];
        float sum = 0.0f;
        if (i >= 0 && i < a.adapters) {
            for (int64_t k = lane; k < a.cols; k += 64)
                sum = fmaf(element(a.x, (size_t)t * (size_t)a.ldx + k), element(a.m, m_at(a, i, j, k)), sum);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
            if (a.scale) sum *= a.scale[i];
        }
        if (lane == 0) a.u[unit] = sum;
    }
}

// One thread: one element.
__global__ __launch_bounds__(256) void adapter_expand(AdapterArgs a, int64_t n) {
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < n; at += (int64_t)gridDim.x * 256) {
        const int t = (int)(at / a.cols);
        const int64_t k = at - (int64_t)t * a.cols;
        const int i = a.index[t];
        float sum = 0.0f;
        if (i >= 0 && i < a.adapters) {
            for (int j = 0; j < a.rank; ++j)
                sum = fmaf(a.u[(size_t)t * a.rank + j], element(a.m, m_at(a, i, j, k)), sum);
            if (a.scale) sum *= a.scale[i];
        }
        static_cast<float*>(a.out)[(size_t)t * (size_t)a.ldo + k] = a.base[(size_t)t * (size_t)a.ld_base + k] + sum;
    }
}

// One thread: one element of one adapter's gradient. Indices from the device are kept inside
// their arrays.
__global__ __launch_bounds__(256) void adapter_gradient(AdapterArgs a, int64_t n) {
    const int64_t each = (int64_t)a.rank * a.cols;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < n; at += (int64_t)gridDim.x * 256) {
        const int i = (int)(at / each);
        const int64_t in = at - i * each;
        const int64_t k = a.turned ? in / a.rank : in % a.cols;
        const int j = (int)(a.turned ? in % a.rank : in / a.cols);
        const int64_t from = max(0, min(a.offsets[i], a.capacity));
        const int64_t to = min((int64_t)a.capacity, from + max(0, a.counts[i]));
        float sum = 0.0f;
        // rows eight at a time, all of their loads before the first product
        int64_t p = from;
        for (; p + 8 <= to; p += 8) {
            float u[8], x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int t = a.rows[p + e];
                const bool in = t >= 0 && t < a.tokens;
                const size_t row = in ? (size_t)t : 0;
                u[e] = a.u[row * a.rank + j];
                x[e] = element(a.x, row * (size_t)a.ldx + k);
                if (!in) u[e] = x[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(u[e], x[e], sum);
        }
        for (; p < to; ++p) {
            const int t = a.rows[p];
            if (t < 0 || t >= a.tokens) continue;
            sum = fmaf(a.u[(size_t)t * a.rank + j], element(a.x, (size_t)t * (size_t)a.ldx + k), sum);
        }
        if (a.scale) sum *= a.scale[i];
        static_cast<float*>(a.out)[at] = sum;
    }
}

namespace {

dim3 walk_grid(int64_t n) {
    const int64_t wgs = (n + 255) / 256;
    return dim3((unsigned)(wgs < (1 << 20) ? wgs : (1 << 20)));
}

}  // namespace

int launch_adapter_shrink(const AdapterArgs& a, hipStream_t s) {
    return launch_status(adapter_shrink, walk_grid((int64_t)a.tokens * a.rank * 64), dim3(256), s, a);
}

int launch_adapter_expand(const AdapterArgs& a, hipStream_t s) {
    const int64_t n = (int64_t)a.tokens * a.cols;
    return launch_status(adapter_expand, walk_grid(n), dim3(256), s, a, n);
}

int launch_adapter_gradient(const AdapterArgs& a, hipStream_t s) {
    const int64_t n = (int64_t)a.adapters * a.rank * a.cols;
    return launch_status(adapter_gradient, walk_grid(n), dim3(256), s, a, n);
}

}  // namespace dg
