// combine.hip -- the weighted sum of each token's expert rows, and its gradients.
//
//   out[t] = sum_j w[t][j] Y[position[t][j]]
//   y_grad[position[t][j]] = w[t][j] G[t]      w_grad[t][j] = G[t] . Y[position[t][j]]
//
// Memory-bound: every row of Y is read once; sums in fp32, in the slots' order.
#include <algorithm>

#include "device_common.h"
#include "experts.h"
#include "launch.h"

namespace dg {

// Eight elements from p, of which `valid` (> 0) exist.
template <int DT>
__device__ __forceinline__ void load8(float (&v)[8], const typename Elem<DT>::type* p, int valid) {
    typename Elem<DT>::type raw[8];
    if (valid >= 8) {
        __builtin_memcpy(raw, p, sizeof raw);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[e] = e < valid ? p[e] : typename Elem<DT>::type(0);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = decode<DT>(raw[e]);
}

template <int DT> __device__ __forceinline__ typename Elem<DT>::type encode(float x);
template <> __device__ __forceinline__ float encode<DT_F32>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t encode<DT_F16>(float x) {
    return __builtin_bit_cast(uint16_t, (_Float16)x);
}
template <> __device__ __forceinline__ uint16_t encode<DT_BF16>(float x) { return f32_to_bf16_rne(x); }

template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::type* p, const float (&v)[8], int valid) {
    typename Elem<DT>::type raw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) raw[e] = encode<DT>(v[e]);
    if (valid >= 8) {
        __builtin_memcpy(p, raw, sizeof raw);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) p[e] = raw[e];
    }
}

// One thread per token and eight columns.
template <int DT>
__global__ __launch_bounds__(256) void combine(CombineArgs a) {
    typedef typename Elem<DT>::type T;
    const int pieces = (a.cols + 2047) >> 11;
    const int64_t total = (int64_t)a.tokens * pieces;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int t = (int)(u / pieces);
        const int c = ((int)(u - (int64_t)t * pieces) * 256 + (int)threadIdx.x) * 8, left = a.cols - c;
        if (left <= 0) continue;
        float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const int* pos = a.position + (size_t)t * a.top_k;
        const float* w = a.weight + (size_t)t * a.top_k;
#pragma unroll 4
        for (int j = 0; j < a.top_k; ++j) {
            const int p = pos[j];
            if (p < 0 || p >= a.capacity) continue;
            float y[8];
            load8<DT>(y, static_cast<const T*>(a.Y) + (size_t)p * (size_t)a.ldy + c, left);
            const float x = w[j];
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = fmaf(x, y[e], sum[e]);
        }
        store8<DT>(static_cast<T*>(a.out) + (size_t)t * (size_t)a.ldo + c, sum, left);
    }
}

// The first `workers` workgroups take a token each in turn, the others clear the padding
// rows of y_grad.
template <int DT>
__global__ __launch_bounds__(256) void combine_backward(CombineArgs a, int workers) {
    typedef typename Elem<DT>::type T;
    __shared__ float dots[kMaxTopK][4];
    const int tid = threadIdx.x;
    T* yg = static_cast<T*>(a.y_grad);
    if ((int)blockIdx.x >= workers) {
        const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int p = (int)blockIdx.x - workers; p < a.capacity; p += (int)gridDim.x - workers) {
            const int r = a.rows[p];
            if (r >= 0 && r < a.tokens) continue;
            for (int c = tid * 8; c < a.cols; c += 2048) store8<DT>(yg + (size_t)p * (size_t)a.ldyg + c, zero, a.cols - c);
        }
        return;
    }
    for (int t = blockIdx.x; t < a.tokens; t += workers) {
        const T* g = static_cast<const T*>(a.G) + (size_t)t * (size_t)a.ldg;
        for (int j = 0; j < a.top_k; ++j) {
            const int p = a.position[(size_t)t * a.top_k + j];
            float dot = 0;
            if (p >= 0 && p < a.capacity) {
                const float w = a.weight[(size_t)t * a.top_k + j];
                const T* y = static_cast<const T*>(a.Y) + (size_t)p * (size_t)a.ldy;
                for (int c = tid * 8; c < a.cols; c += 2048) {
                    float gv[8], yv[8];
                    load8<DT>(gv, g + c, a.cols - c);
                    load8<DT>(yv, y + c, a.cols - c);
    #pragma unroll
                    for (int e = 0; e < 8; ++e) dot = fmaf(gv[e], yv[e], dot);
    #pragma unroll
                    for (int e = 0; e < 8; ++e) gv[e] *= w;
                    store8<DT>(yg + (size_t)p * (size_t)a.ldyg + c, gv, a.cols - c);
                }
            }
    #pragma unroll
            for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
            if ((tid & 63) == 0) dots[j][tid >> 6] = dot;
        }
        __syncthreads();
        if (tid < a.top_k) a.weight_grad[(size_t)t * a.top_k + tid] = (dots[tid][0] + dots[tid][1]) + (dots[tid][2] + dots[tid][3]);
        __syncthreads();
    }
}

int launch_combine(const CombineArgs& a, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)std::min<int64_t>((int64_t)a.tokens * ((a.cols + 2047) / 2048), 1 << 20));
    if (dtype == DT_F32) return launch_status(combine<DT_F32>, grid, dim3(256), s, a);
    if (dtype == DT_F16) return launch_status(combine<DT_F16>, grid, dim3(256), s, a);
    return launch_status(combine<DT_BF16>, grid, dim3(256), s, a);
}

int launch_combine_backward(const CombineArgs& a, int dtype, hipStream_t s) {
    const int64_t spare = (int64_t)a.capacity - (int64_t)a.tokens * a.top_k;
    const int clear = spare > 0 ? (int)std::min<int64_t>(a.capacity, 2048) : 0;
    const int workers = std::min(a.tokens, 1 << 20);
    const dim3 grid((unsigned)(workers + std::max(clear, 1)));
    if (dtype == DT_F32) return launch_status(combine_backward<DT_F32>, grid, dim3(256), s, a, workers);
    if (dtype == DT_F16) return launch_status(combine_backward<DT_F16>, grid, dim3(256), s, a, workers);
    return launch_status(combine_backward<DT_BF16>, grid, dim3(256), s, a, workers);
}

}  // namespace dg
