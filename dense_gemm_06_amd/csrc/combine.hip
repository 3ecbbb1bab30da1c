// combine.hip -- the weighted sum of each token's expert rows, and its gradients.
//
//   out[t] = sum_j w[t][j] Y[position[t][j]]
//   y_grad[position[t][j]] = w[t][j] G[t]      w_grad[t][j] = G[t] . Y[position[t][j]]
//
// Memory-bound: every row of Y is read once; sums in fp32, in the slots' order. 4096 tokens
// x 8 rows of 4096 bf16: 300 MB in 55 to 78 us forward (5.5 to 3.9 TB/s, with Y partly in
// the caches or not), 637 MB in 112 us backward (5.7 TB/s; 67 MB of it zeros of padding rows).
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "experts.h"
#include "extents.h"
#include "launch.h"

namespace dg {

// Eight elements from p, of which `valid` (> 0) exist (the rest zero).
template <int DT>
__device__ __forceinline__ void load8_raw(typename Elem<DT>::type (&raw)[8], const typename Elem<DT>::type* p, int valid) {
    if (valid >= 8) {
        __builtin_memcpy(raw, p, sizeof raw);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[e] = e < valid ? p[e] : typename Elem<DT>::type(0);
    }
}

template <int DT> __device__ __forceinline__ typename Elem<DT>::type encode(float x);
template <> __device__ __forceinline__ float encode<DT_F32>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t encode<DT_F16>(float x) {
    return __builtin_bit_cast(uint16_t, (_Float16)x);
}
template <> __device__ __forceinline__ uint16_t encode<DT_BF16>(float x) { return f32_to_bf16_rne(x); }

// PASSING: y_grad, whose stores go past the caches: 300 MB that would take Y and G out of them.
// 4096 tokens x 8 rows of 4096 bf16, both directions: 180 us against 203; with the gradient
// quantized right behind, 277 against 276 (38 against 39 for 128 tokens x 4 rows of 2048). out
// is small and read next, so it stays.
template <int DT, bool PASSING = false>
__device__ __forceinline__ void store8(typename Elem<DT>::type* p, const float (&v)[8], int valid) {
    typename Elem<DT>::type raw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) raw[e] = encode<DT>(v[e]);
    if (valid >= 8) {
        if constexpr (PASSING) {
#pragma unroll
            for (int e = 0; e < 8; e += 16 / (int)sizeof raw[0]) {
                u32x4 q;
                __builtin_memcpy(&q, raw + e, 16);
                store_passing(p + e, q);
            }
        } else {
            __builtin_memcpy(p, raw, sizeof raw);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) p[e] = raw[e];
    }
}

// Slots are taken eight at a time, their rows' loads all in flight together: a slot's row
// and weight are the same for a whole workgroup, a slot without a row reads row 0 and drops
// what it read.
constexpr int kSlots = 8;

struct Slots {
    int p[kSlots];
    float w[kSlots];
    bool in[kSlots];
};

__device__ __forceinline__ Slots slots_of(const CombineArgs& a, int t, int j0) {
    Slots s;
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
        const size_t at = (size_t)t * a.top_k + min(j0 + u, a.top_k - 1);
        const int p = a.position[at];
        s.in[u] = j0 + u < a.top_k && p >= 0 && p < a.capacity;
        s.p[u] = s.in[u] ? p : 0;
        s.w[u] = a.weight[at];
    }
    return s;
}

// One workgroup per token, eight columns to a thread and 2048 to a pass. (Two workgroups to
// a token of 4096 columns, with half rows each: 90 us against 86 at 4096 tokens x 8 rows.)
template <int DT>
__global__ __launch_bounds__(256) void combine(CombineArgs a) {
    typedef typename Elem<DT>::type T;
    stride_walk(blockIdx.x, a.tokens, gridDim.x, [&](int t) {
        auto piece = [&](int c, auto whole_tag) {
            const int left = decltype(whole_tag)::value ? 8 : a.cols - c;
            float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (a.capacity > 0)
                stride_walk(0, a.top_k, kSlots, [&](int j0) {
                    const Slots s = slots_of(a, t, j0);
                    T raw[kSlots][8];
#pragma unroll
                    for (int v = 0; v < kSlots; ++v)
                        load8_raw<DT>(raw[v], static_cast<const T*>(a.Y) + (size_t)s.p[v] * (size_t)a.ldy + c, left);
#pragma unroll
                    for (int v = 0; v < kSlots; ++v)
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum[e] = s.in[v] ? fmaf(s.w[v], decode<DT>(raw[v][e]), sum[e]) : sum[e];
                });
            store8<DT>(static_cast<T*>(a.out) + (size_t)t * (size_t)a.ldo + c, sum, left);
        };
        // whole passes without a branch at each load
        int c0 = 0;
        for (; a.cols - c0 >= 2048; c0 += 2048) piece(c0 + (int)threadIdx.x * 8, std::true_type{});
        if ((int)threadIdx.x * 8 < a.cols - c0) piece(c0 + (int)threadIdx.x * 8, std::false_type{});
    });
}

// The first `workers` workgroups take a token each in turn, the others clear the padding
// rows of y_grad.
template <int DT>
__global__ __launch_bounds__(256) void combine_backward(CombineArgs a, int workers) {
    typedef typename Elem<DT>::type T;
    __shared__ float dots[kSlots][4];
    const int tid = threadIdx.x;
    T* yg = static_cast<T*>(a.y_grad);
    if ((int)blockIdx.x >= workers) {
        // 4 rows at a time, looked through by every wave alike (one row after the other cost a
        // lone workgroup 160 us for 1604 rows without padding)
        const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const int64_t step = (int64_t)((int)gridDim.x - workers) * 4;
        for (int64_t p0 = (int64_t)((int)blockIdx.x - workers) * 4; p0 < a.capacity; p0 += step) {
            const int64_t p = p0 + (tid & 3);
            const int r = p < a.capacity ? a.rows[p] : 0;
            for (uint64_t pad = __ballot(p < a.capacity && (r < 0 || r >= a.tokens)) & 0xf; pad; pad &= pad - 1) {
                T* const row = yg + (size_t)(p0 + __builtin_ctzll(pad)) * (size_t)a.ldyg;
                stride_walk(tid * 8, a.cols, 2048, [&](int c) { store8<DT, true>(row + c, zero, a.cols - c); });
            }
        }
        return;
    }
    stride_walk(blockIdx.x, a.tokens, workers, [&](int t) {
        const T* g = static_cast<const T*>(a.G) + (size_t)t * (size_t)a.ldg;
        for (int j0 = 0; j0 < a.top_k; j0 += kSlots) {
            const Slots s = slots_of(a, t, j0);
            float dot[kSlots] = {0, 0, 0, 0, 0, 0, 0, 0};
            auto piece = [&](int c, auto whole_tag) {
                const int left = decltype(whole_tag)::value ? 8 : a.cols - c;
                T raw[kSlots][8], graw[8];
                load8_raw<DT>(graw, g + c, left);
                if (a.capacity > 0)
#pragma unroll
                    for (int v = 0; v < kSlots; ++v)
                        load8_raw<DT>(raw[v], static_cast<const T*>(a.Y) + (size_t)s.p[v] * (size_t)a.ldy + c, left);
#pragma unroll
                for (int v = 0; v < kSlots; ++v) {
                    if (!s.in[v]) continue;
                    float out[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float x = decode<DT>(graw[e]);
                        dot[v] = fmaf(x, decode<DT>(raw[v][e]), dot[v]);
                        out[e] = x * s.w[v];
                    }
                    store8<DT, true>(yg + (size_t)s.p[v] * (size_t)a.ldyg + c, out, left);
                }
            };
            int c0 = 0;
            for (; a.cols - c0 >= 2048; c0 += 2048) piece(c0 + tid * 8, std::true_type{});
            if (tid * 8 < a.cols - c0) piece(c0 + tid * 8, std::false_type{});
#pragma unroll
            for (int v = 0; v < kSlots; ++v) {
#pragma unroll
                for (int d = 32; d; d >>= 1) dot[v] += __shfl_xor(dot[v], d);
                if ((tid & 63) == 0) dots[v][tid >> 6] = dot[v];
            }
            __syncthreads();
            if (tid < kSlots && j0 + tid < a.top_k)
                a.weight_grad[(size_t)t * a.top_k + j0 + tid] =
                    (dots[tid][0] + dots[tid][1]) + (dots[tid][2] + dots[tid][3]);
            __syncthreads();
        }
    });
}

int launch_combine(const CombineArgs& a, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)std::min(a.tokens, 1 << 20));
    if (dtype == DT_F32) return launch_status(combine<DT_F32>, grid, dim3(256), s, a);
    if (dtype == DT_F16) return launch_status(combine<DT_F16>, grid, dim3(256), s, a);
    return launch_status(combine<DT_BF16>, grid, dim3(256), s, a);
}

int launch_combine_backward(const CombineArgs& a, int dtype, hipStream_t s) {
    const int workers = std::min(a.tokens, 1 << 20), clear = (int)std::max<int64_t>(1, std::min<int64_t>(((int64_t)a.capacity + 3) / 4, 16384));
    const dim3 grid((unsigned)(workers + clear));
    if (dtype == DT_F32) return launch_status(combine_backward<DT_F32>, grid, dim3(256), s, a, workers);
    if (dtype == DT_F16) return launch_status(combine_backward<DT_F16>, grid, dim3(256), s, a, workers);
    return launch_status(combine_backward<DT_BF16>, grid, dim3(256), s, a, workers);
}

}  // namespace dg
