// adapters.hip -- low-rank adapters of many requests beside a shared product, in fp32.
//
//   u[t] = scale a_i x[t]      (shrink)        out[t] = base[t] + scale b_i u[t]   (expand)
//   a_grad_i = sum_t v[t] x[t]^T over adapter i's rows                             (gradient)
//
// The same kernels serve the backward pass with the roles of a and b exchanged, which differ
// in the direction that lies along memory (`turned`). fp32 has no fast matrix instructions, and the
// adapters' own work is small beside the shared product, so vector instructions do it. Bound by latency:
// each launch takes 8 to 9 us (512 tokens, 1024 x 1024, rank 12, 3 adapters, both ways: 70 us with the
// shared products' 39; four rank numbers to a wave, read together where they are neighbours: 6 us more).
#include "device_common.h"
#include "extents.h"
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

// One wave: one token and one of its rank numbers (four to a workgroup, along grid y).
__global__ __launch_bounds__(256) void adapter_shrink(AdapterArgs a) {
    const int lane = threadIdx.x & 63, j = (int)blockIdx.y * 4 + (int)(threadIdx.x >> 6);
    if (j >= a.rank) return;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const int i = a.index[t];
        float sum = 0.0f;
        if (i >= 0 && i < a.adapters) {
            const float* x = static_cast<const float*>(a.x) + (size_t)t * (size_t)a.ldx;
            const float* m = static_cast<const float*>(a.m) + m_at(a, i, j, 0);
            const int64_t step = a.turned ? a.ldm : 1;
#pragma unroll 8
            for (int64_t k = lane; k < a.cols; k += 64) sum = fmaf(x[k], m[k * step], sum);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
            if (a.scale) sum *= a.scale[i];
        }
        if (lane == 0) a.u[(size_t)t * a.rank + j] = sum;
    }
}

// One thread: one element, columns along grid x and tokens along grid y.
__global__ __launch_bounds__(256) void adapter_expand(AdapterArgs a) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= a.cols) return;
    for (int64_t t = blockIdx.y; t < a.tokens; t += gridDim.y) {
        const int i = a.index[t];
        float sum = 0.0f;
        if (i >= 0 && i < a.adapters) {
            const float* u = a.u + (size_t)t * a.rank;
            const float* m = static_cast<const float*>(a.m) + m_at(a, i, 0, k);
            const int64_t step = a.turned ? 1 : a.ldm;
#pragma unroll 8
            for (int j = 0; j < a.rank; ++j) sum = fmaf(u[j], m[j * step], sum);
            if (a.scale) sum *= a.scale[i];
        }
        static_cast<float*>(a.out)[(size_t)t * (size_t)a.ldo + k] = a.base[(size_t)t * (size_t)a.ld_base + k] + sum;
    }
}

// One workgroup: 64 columns and 16 rank numbers of one adapter's gradient, its rows shared out over the
// waves, eight at a time with all of their loads before the first product, and the waves' sums joined in
// order. Indices from the device are kept inside their arrays.
constexpr int kGradWaves = 8, kGradRank = 16;
__device__ __forceinline__ void gradient_block(const AdapterArgs& a, int block, float (*part)[kGradRank][64]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t k = (int64_t)block * 64 + lane;
    const int i = (int)blockIdx.z, j0 = (int)blockIdx.y * kGradRank;
    const int64_t from = max(0, min(a.offsets[i], a.capacity));
    const int64_t to = min((int64_t)a.capacity, from + max(0, a.counts[i]));
    const bool in_cols = k < a.cols;
    const int64_t column = in_cols ? k : 0;
    float sum[kGradRank];
#pragma unroll
    for (int j = 0; j < kGradRank; ++j) sum[j] = 0.0f;
    for (int64_t p = from + wave * 8; p < to; p += 8 * kGradWaves) {
        // lane 8 e + j has rank numbers j and j + 8 of row e, and hands them round
        const float* xs = static_cast<const float*>(a.x);
        const int mine = p + (lane >> 3) < to ? a.rows[p + (lane >> 3)] : -1;
        const bool in = mine >= 0 && mine < a.tokens;
        float x[8], u[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = j0 + 8 * h + (lane & 7);
            u[h] = in && j < a.rank ? a.u[(size_t)mine * a.rank + j] : 0.0f;
        }
        const uint64_t rows_in = __ballot(in);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = rows_in >> (8 * e) & 1 ? __builtin_amdgcn_readlane(mine, 8 * e) : 0;
            x[e] = xs[(size_t)t * (size_t)a.ldx + column];
            if (!(rows_in >> (8 * e) & 1)) x[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int j = 0; j < kGradRank; ++j) {
                const int one = __builtin_amdgcn_readlane(__float_as_int(u[j >> 3]), 8 * e + (j & 7));
                sum[j] = fmaf(__int_as_float(one), x[e], sum[j]);
            }
    }
#pragma unroll
    for (int j = 0; j < kGradRank; ++j) part[wave][j][lane] = sum[j];
    __syncthreads();
    for (int j = wave; j < kGradRank; j += kGradWaves) {
        if (j0 + j >= a.rank || !in_cols) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kGradWaves; ++w) v += part[w][j][lane];
        if (a.scale) v *= a.scale[i];
        const size_t at = (size_t)i * (size_t)a.rank * (size_t)a.cols +
                          (a.turned ? (size_t)k * a.rank + j0 + j : (size_t)(j0 + j) * a.cols + k);
        static_cast<float*>(a.out)[at] = v;
    }
}

// Both gradients in one launch: the first blocks along grid x are a's.
__global__ __launch_bounds__(64 * kGradWaves) void adapter_gradient(AdapterArgs a, AdapterArgs b, int blocks) {
    __shared__ float part[kGradWaves][kGradRank][64];
    if ((int)blockIdx.x < blocks) gradient_block(a, (int)blockIdx.x, part);
    else gradient_block(b, (int)blockIdx.x - blocks, part);
}

int launch_adapter_shrink(const AdapterArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.tokens < (1 << 20) ? a.tokens : (1 << 20)), (unsigned)((a.rank + 3) / 4));
    return launch_status(adapter_shrink, grid, dim3(256), s, a);
}

int launch_adapter_expand(const AdapterArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(((int64_t)a.cols + 255) / 256), (unsigned)(a.tokens < 32768 ? a.tokens : 32768));
    return launch_status(adapter_expand, grid, dim3(256), s, a);
}

int launch_adapter_gradient(const AdapterArgs& a, const AdapterArgs& b, hipStream_t s) {
    const int blocks = pieces<64>(a.cols);
    const dim3 grid((unsigned)(blocks + pieces<64>(b.cols)), (unsigned)pieces<kGradRank>(a.rank), (unsigned)a.adapters);
    return launch_status(adapter_gradient, grid, dim3(64 * kGradWaves), s, a, b, blocks);
}

}  // namespace dg
