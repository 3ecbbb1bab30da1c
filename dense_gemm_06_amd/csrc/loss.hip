// loss.hip -- softmax cross entropy over a vocabulary whose logits are made a piece of the
// vocabulary at a time.
//
// A row's running maximum m and sum s of exp(l - m) take a piece's own (m', s') in as
//   M = max(m, m'),  s = s exp(m - M) + s' exp(m' - M),
// so one pass over the pieces gives lse = m + log(s).
#include "device_common.h"
#include "layers.h"
#include "launch.h"

namespace dg {

namespace {

// (m, s) joined with (m2, s2); a part without anything is (-inf, 0).
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float M = fmaxf(m, m2);
    const float a = m == M ? 1.0f : __expf(m - M), b = m2 == M ? 1.0f : __expf(m2 - M);
    s = s * a + s2 * b;
    m = M;
}

}  // namespace

// One workgroup: a row's part of the piece (1000 x 8192: 8.2 us, 4 TB/s).
__global__ __launch_bounds__(256) void loss_stats(LossArgs a) {
    __shared__ float part[2][4];
    const int t = blockIdx.x, tid = threadIdx.x;
    const float* l = a.logits + (size_t)t * (size_t)a.ld;
    float m = -INFINITY, s = 0.0f;
    // eight at a time, all loaded before the first is used, for one change of the maximum
    for (int64_t j = tid; j < a.n; j += 8 * 256) {
        float v[8], top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = j + 256 * e < a.n ? l[min(j + 256 * e, (int64_t)a.n - 1)] : -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, v[e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += v[e] == top ? 1.0f : __expf(v[e] - top);
        join(m, s, top, sum);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float m2 = __shfl_xor(m, d), s2 = __shfl_xor(s, d);
        join(m, s, m2, s2);
    }
    if ((tid & 63) == 0) {
        part[0][tid >> 6] = m;
        part[1][tid >> 6] = s;
    }
    __syncthreads();
    if (tid != 0) return;
#pragma unroll
    for (int w = 1; w < 4; ++w) join(m, s, part[0][w], part[1][w]);
    float picked = a.first ? 0.0f : a.picked[t];
    if (!a.first) join(m, s, a.top[t], a.sum[t]);
    const int64_t target = a.target[t];
    if (target >= a.v0 && target < (int64_t)a.v0 + a.n) picked = l[target - a.v0];
    if (!a.last) {
        a.top[t] = m;
        a.sum[t] = s;
        a.picked[t] = picked;
        return;
    }
    const float lse = m + logf(s);
    a.lse[t] = lse;
    a.loss[t] = target >= 0 && target < a.vocabulary ? lse - picked : 0.0f;
}

// One workgroup: 64 x 64 of the piece. Rows past the last token are zeros in the transpose. All
// loads come first (1000 x 8192: 17 us, 5.8 TB/s; row by row 20, and 200 x 4000 13 us against 6.6).
template <int DT>
__global__ __launch_bounds__(256) void loss_grad(LossArgs a, int tiles_n) {
    __shared__ float turned[64][65];
    const int tm = (int)blockIdx.x / tiles_n, tn = (int)blockIdx.x - tm * tiles_n;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t j = (int64_t)tn * 64 + lane;
    // lane i of a wave has row i's numbers and hands them round
    const int64_t own = min((int64_t)tm * 64 + lane, (int64_t)a.tokens - 1), own_target = a.target[own];
    const float own_grad = a.factor ? a.grad[own] * a.factor[0] : a.grad[own], own_lse = a.lse_in[own];
    const bool own_live = own_target >= 0 && own_target < a.vocabulary && own_grad != 0.0f;
    const int own_at = own_live ? (int)own_target : -1;
    float l[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int64_t t = min((int64_t)tm * 64 + wave + 4 * e, (int64_t)a.tokens - 1);
        l[e] = a.logits[(size_t)t * (size_t)a.ld + min(j, (int64_t)a.n - 1)];
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int i = wave + 4 * e, target = __shfl(own_at, i);
        const float g = __shfl(own_grad, i), lse = __shfl(own_lse, i);
        const int64_t t = (int64_t)tm * 64 + i;
        float d = 0.0f;
        if (t < a.tokens && j < a.n) {
            if (target >= 0) d = (__expf(l[e] - lse) - (target == a.v0 + j ? 1.0f : 0.0f)) * g;
            if (a.d) store_out(a.d, DT, (size_t)t * (size_t)a.ldd + j, d);
        }
        turned[lane][i] = d;
    }
    if (a.dt == nullptr) return;
    __syncthreads();
#pragma unroll
    for (int i = wave; i < 64; i += 4) {
        const int64_t v = (int64_t)tn * 64 + i, t = (int64_t)tm * 64 + lane;
        if (v < a.n && t < a.lddt) store_out(a.dt, DT, (size_t)v * (size_t)a.lddt + t, turned[i][lane]);
    }
}

// One workgroup: the largest finite |grad| as a power of two 2^e, factor = 2^(14 - e), 2^(e - 14).
__global__ __launch_bounds__(256) void loss_factor(const float* grad, int tokens, float* factor) {
    __shared__ uint32_t part[4];
    uint32_t m = 0;
    for (int64_t t = threadIdx.x; t < tokens; t += 256) {
        const uint32_t u = __float_as_uint(grad[t]) & 0x7fffffffu;
        if (u < 0x7f800000u) m = max(m, u);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x != 0) return;
    m = max(max(part[0], part[1]), max(part[2], part[3]));
    // within 2^-100 .. 2^100, so that both factors are normal numbers
    const int e = m == 0 ? 0 : min(max((int)(m >> 23) - 126, -100), 100);
    factor[0] = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    factor[1] = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
}

// out = in factor[1] - apart[t] grad[t] w[target[t]] for x's gradient (w NULL: without the second
// term). Four columns of a row to a thread, rows over grid y.
template <int DT>
__global__ __launch_bounds__(256) void scaled_cast(const float* in, int64_t ldi, int rows, int cols,
                                                   const float* factor, void* out, int64_t ldo, const void* w,
                                                   int64_t ldw, const int64_t* target, int vocabulary,
                                                   const float* grad, const float* apart) {
    const float f = factor ? factor[1] : 1.0f;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    const int left = (int)min((int64_t)4, cols - c);
    if (left <= 0) return;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float* src = in + (size_t)r * (size_t)ldi + c;
        const size_t at = (size_t)r * (size_t)ldo + c;
        float g = 0.0f;
        size_t row = 0;
        if (w) {
            const int64_t t = target[r];
            if (t >= 0 && t < vocabulary && grad[r] != 0.0f && apart[r] != 0.0f) {
                g = grad[r];
                row = (size_t)t * (size_t)ldw + c;
            }
        }
        if (left == 4) {
            f32x4 v;
            __builtin_memcpy(&v, src, 16);
            v = v * f;
            if (g != 0.0f) {
                const f32x4 h = load_out4(w, DT, row);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = fmaf(-g, h[e], v[e]);
            }
            store_out4(out, DT, at, v);
        } else {
            for (int e = 0; e < left; ++e) {
                const float v = src[e] * f;
                store_out(out, DT, at + e, g != 0.0f ? fmaf(-g, load_out(w, DT, row + e), v) : v);
            }
        }
    }
}

int launch_loss_stats(const LossArgs& a, hipStream_t s) {
    return launch_status(loss_stats, dim3((unsigned)a.tokens), dim3(256), s, a);
}

int launch_loss_grad(const LossArgs& a, int dtype, hipStream_t s) {
    const int tiles_n = (a.n + 63) / 64;
    const dim3 grid((unsigned)(((int64_t)a.tokens + 63) / 64 * tiles_n));
    if (dtype == DT_F32) return launch_status(loss_grad<DT_F32>, grid, dim3(256), s, a, tiles_n);
    if (dtype == DT_F16) return launch_status(loss_grad<DT_F16>, grid, dim3(256), s, a, tiles_n);
    return launch_status(loss_grad<DT_BF16>, grid, dim3(256), s, a, tiles_n);
}

int launch_loss_factor(const float* grad, int tokens, float* factor, hipStream_t s) {
    return launch_status(loss_factor, dim3(1), dim3(256), s, grad, tokens, factor);
}

int launch_scaled_cast(const float* in, int64_t ldi, int rows, int cols, const float* factor, void* out, int64_t ldo,
                       const void* w, int64_t ldw, const int64_t* target, int vocabulary, const float* grad,
                       const float* apart, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)(((int64_t)cols + 1023) / 1024), (unsigned)(rows < 32768 ? rows : 32768));
    return dtype == DT_F16 ? launch_status(scaled_cast<DT_F16>, grid, dim3(256), s, in, ldi, rows, cols, factor, out, ldo,
                                           w, ldw, target, vocabulary, grad, apart)
                           : launch_status(scaled_cast<DT_BF16>, grid, dim3(256), s, in, ldi, rows, cols, factor, out, ldo,
                                           w, ldw, target, vocabulary, grad, apart);
}

}  // namespace dg
