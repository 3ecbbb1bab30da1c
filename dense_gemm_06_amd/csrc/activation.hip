// activation.hip -- activations whose input is kept in 8 bits, and their backward pass from
// the codes.
//
//   y = f(z), or f(z1) z2 with z = [z1 | z2]; codes and scales of z over blocks of 1 x 128
//   z_grad = g f'(z), or [g z2 f'(z1) | g f(z1)], z being the codes' values
//
// With e = exp(-v) and s = 1 / (1 + e), silu is v s and its slope s (1 + v e s); gelu in its
// tanh form is v s with e = exp(-2w), w = sqrt(2/pi) (v + 0.044715 v^3), and its slope
// s + v e s^2 (2w)'. 1 - s = e s keeps its digits where s is near 1.
//
// 16 lanes hold a block of 128, eight values each: a block's maximum takes four exchanges, a
// block's codes leave as a whole 128-byte line.
#include "device_common.h"
#include "extents.h"
#include "layers.h"
#include "launch.h"

namespace dg {

namespace {

// e^x: the product x log2(e) with its rounding error put back, so that the relative error
// does not grow with |x|.
__device__ __forceinline__ float exp_exact(float x) {
    const float hi = 1.44269502f, lo = 1.92596303e-8f;
    const float t = x * hi;
    float e = fmaf(x, lo, fmaf(x, hi, -t));
    e = fabsf(t) < 256.0f ? e : 0.0f;
    return __builtin_amdgcn_exp2f(t) * fmaf(e, 0.693147182f, 1.0f);
}

// f(v) and, with SLOPE, f'(v)
template <bool SLOPE>
__device__ __forceinline__ void act_value(float v, int act, float& f, float& slope) {
    if (act == ACT_RELU) {
        f = v <= 0.0f ? 0.0f : v;  // a NaN stays one
        slope = v > 0.0f ? 1.0f : f;
        return;
    }
    const bool gelu = act == ACT_GELU_TANH;
    const float w2 = gelu ? 1.5957691216057308f * fmaf(0.044715f * v * v, v, v) : v;
    const float e = exp_exact(-w2);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    f = v * s;
    if (SLOPE) {
        // where e overflows s is 0, and so is the slope
        const float c = v * (fminf(e, 1e30f) * s);
        // past 2^40 c is 0, and v^2 must not be infinite
        const float q = fminf(fabsf(v), 1.09951163e12f);
        slope = gelu ? fmaf(c * s, 1.5957691216057308f * fmaf(0.134145f * q, q, 1.0f), s) : s * (1.0f + c);
    }
}

// N 16-byte pieces at any address, past the caches with PASSING (no branch at run time:
// one took half of the gain).
template <int N, bool PASSING>
__device__ __forceinline__ void load_pieces(void* to, const void* from) {
    typedef u32x4 any_address __attribute__((aligned(1)));
    if (!PASSING) {
        __builtin_memcpy(to, from, 16 * N);
    } else {
        u32x4 q[N];
#pragma unroll
        for (int k = 0; k < N; ++k) q[k] = __builtin_nontemporal_load(static_cast<const any_address*>(from) + k);
        __builtin_memcpy(to, q, sizeof q);
    }
}

template <int DT, bool PASSING>
__device__ __forceinline__ void load_row8(float (&v)[8], const void* p, size_t at, int valid) {
    typedef typename Elem<DT>::type T;
    const T* src = static_cast<const T*>(p) + at;
    T raw[8];
    if (valid >= 8) {
        load_pieces<sizeof raw / 16, PASSING>(raw, src);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[e] = e < valid ? src[e] : T(0);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = decode<DT>(raw[e]);
}

// Eight results: past the caches where all of them together would not stay there (PASSING), as
// one store of 16 bytes; else as two stores, since one made the whole pass 10% slower.
template <int DT, bool PASSING>
__device__ __forceinline__ void store_row8(void* p, size_t at, const float (&v)[8], int valid) {
    if (valid >= 8) {
        if constexpr (!PASSING) {
            store_out4(p, DT, at, f32x4{v[0], v[1], v[2], v[3]});
            store_out4(p, DT, at + 4, f32x4{v[4], v[5], v[6], v[7]});
        } else if constexpr (DT == DT_F32) {
            store_passing(static_cast<float*>(p) + at, f32x4{v[0], v[1], v[2], v[3]});
            store_passing(static_cast<float*>(p) + at + 4, f32x4{v[4], v[5], v[6], v[7]});
        } else {
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[e] = DT == DT_F16 ? (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[e]) : (uint32_t)f32_to_bf16_rne(v[e]);
            store_passing(static_cast<uint16_t*>(p) + at, u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16),
                                                                h[4] | (h[5] << 16), h[6] | (h[7] << 16)});
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) store_out(p, DT, at + e, v[e]);
    }
}

// The codes and the scale of block `blk` of a row, of which this lane holds the eight values
// at column c (`valid` of them inside the row): as block_quantize.
__device__ __forceinline__ void quantize_block(const QuantOut& o, const float (&v)[8], int row, int blk, int c,
                                               int valid) {
    uint32_t m = (127u - 100u) << 23;  // 2^-100
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    const float top = o.type == 0 ? 448.0f : 57344.0f, amax = __uint_as_float(m), inv = top / amax;
    uint32_t q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int r = 0;
        const float a = v[4 * h] * inv, b = v[4 * h + 1] * inv, c2 = v[4 * h + 2] * inv, d = v[4 * h + 3] * inv;
        if (o.type == 0) {
            r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
            r = __builtin_amdgcn_cvt_pk_fp8_f32(c2, d, r, true);
        } else {
            r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
            r = __builtin_amdgcn_cvt_pk_bf8_f32(c2, d, r, true);
        }
        q[h] = (uint32_t)r;
    }
    uint8_t* dst = o.q + (size_t)row * (size_t)o.ld + c;
    if (valid >= 8) {
        __builtin_memcpy(dst, q, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) dst[e] = (uint8_t)(q[e >> 2] >> (8 * (e & 3)));
    }
    if ((threadIdx.x & 15) == 0) o.s[(size_t)row * (size_t)o.s_row + (size_t)blk * (size_t)o.s_blk] = amax / top;
}

// The unit of 16 lanes: row and number within the row's `per` units. A workgroup's first unit
// is divided once; its others are a few steps on.
__device__ __forceinline__ void unit_of(int64_t first, int per, int& row, int& k) {
    const int64_t r0 = first / per;
    const uint32_t step = (uint32_t)(first - r0 * per) + (threadIdx.x >> 4);
    const uint32_t more = step / (uint32_t)per;
    row = (int)(r0 + more);
    k = (int)(step - more * (uint32_t)per);
}

}  // namespace

// A unit is a block of 128 columns of y with the block(s) of z behind it. Where the second
// half of z does not start with a block (SPLIT), a row's units are first the blocks of z,
// which only make codes, and then the blocks of y.
template <int DT, bool SPLIT, bool PASSING>
__global__ __launch_bounds__(256) void activation_forward(ActArgs a, int64_t units, int per) {
    const int zcols = a.gated ? 2 * a.cols : a.cols;
    const int zblocks = SPLIT ? pieces<128>(zcols) : 0;
    const int groups = (int)blockDim.x >> 4, g = (int)threadIdx.x >> 4;
    for (int64_t first = (int64_t)blockIdx.x * groups; first < units; first += (int64_t)gridDim.x * groups) {
        if (first + g >= units) return;  // 16 lanes leave together, and only they work together
        int row, k;
        unit_of(first, per, row, k);
        const bool code_unit = SPLIT && k < zblocks;
        const int blk = SPLIT && !code_unit ? k - zblocks : k;
        const int width = code_unit ? zcols : a.cols;
        const int64_t c64 = (int64_t)blk * 128 + (threadIdx.x & 15) * 8;
        const int valid = c64 < width ? (int)(width - c64) : 0, c = valid > 0 ? (int)c64 : 0;
        const size_t zrow = (size_t)row * (size_t)a.ldz;
        float v[8], w[8];
        load_row8<DT, PASSING>(v, a.z, zrow + c, valid);
        if (a.gated && !code_unit) load_row8<DT, PASSING>(w, a.z, zrow + a.cols + c, valid);
        if (!code_unit) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float slope;
                act_value<false>(v[e], a.act, y[e], slope);
                if (a.gated) y[e] *= w[e];
            }
            store_row8<DT, PASSING>(a.y, (size_t)row * (size_t)a.ldy + c, y, valid);
        }
        if (a.codes.q == nullptr) continue;
        if (!SPLIT || code_unit) quantize_block(a.codes, v, row, blk, c, valid);
        if (!SPLIT && a.gated) quantize_block(a.codes, w, row, blk + (a.cols >> 7), a.cols + c, valid);
    }
}

// Eight values of a row from codes and scales, the first at column c: they lie in one block
// or in two neighbouring ones.
__device__ __forceinline__ void decode_row8(float (&v)[8], const QuantOut& o, int row, int c, int valid, int zcols) {
    const uint8_t* src = o.q + (size_t)row * (size_t)o.ld + c;
    uint32_t q[2] = {0, 0};
    if (valid >= 8) {
        __builtin_memcpy(q, src, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) q[e >> 2] |= (uint32_t)src[e] << (8 * (e & 3));
    }
    const int b0 = c >> 7, b1 = (valid >= 8 ? c + 7 : zcols - 1) >> 7;
    const float* s = o.s + (size_t)(o.block_rows == 1 ? row : row >> 7) * (size_t)o.s_row;
    const float s0 = s[(size_t)b0 * (size_t)o.s_blk];
    const float s1 = b1 > b0 ? s[(size_t)(b0 + 1) * (size_t)o.s_blk] : s0;
    const int edge = 128 - (c & 127);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const int word = (int)q[h >> 1];
        f32x2 p;
        if (o.type == 0)
            p = (h & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8(word, true) : __builtin_amdgcn_cvt_pk_f32_fp8(word, false);
        else
            p = (h & 1) ? __builtin_amdgcn_cvt_pk_f32_bf8(word, true) : __builtin_amdgcn_cvt_pk_f32_bf8(word, false);
        v[2 * h] = p[0] * (2 * h < edge ? s0 : s1);
        v[2 * h + 1] = p[1] * (2 * h + 1 < edge ? s0 : s1);
    }
}

template <int DT, bool PASSING>
__global__ __launch_bounds__(256) void activation_backward(ActArgs a, int64_t units, int per) {
    const int zcols = a.gated ? 2 * a.cols : a.cols;
    const int groups = (int)blockDim.x >> 4, g = (int)threadIdx.x >> 4;
    for (int64_t first = (int64_t)blockIdx.x * groups; first < units; first += (int64_t)gridDim.x * groups) {
        if (first + g >= units) return;
        int row, blk;
        unit_of(first, per, row, blk);
        const int64_t c64 = (int64_t)blk * 128 + (threadIdx.x & 15) * 8;
        if (c64 >= a.cols) continue;
        const int c = (int)c64, valid = a.cols - c;
        float v[8], w[8], gr[8], z1[8], z2[8], y[8];
        if (a.grad) load_row8<DT, PASSING>(gr, a.grad, (size_t)row * (size_t)a.ldg + c, valid);
        decode_row8(v, a.codes, row, c, valid, a.cols);
        if (a.gated) decode_row8(w, a.codes, row, a.cols + c, valid, zcols);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float f, slope;
            act_value<true>(v[e], a.act, f, slope);
            if (a.grad == nullptr) gr[e] = 0.0f;
            if (a.gated) {
                z1[e] = gr[e] * w[e] * slope;
                z2[e] = gr[e] * f;
                y[e] = f * w[e];
            } else {
                z1[e] = gr[e] * slope;
                y[e] = f;
            }
        }
        const size_t at = (size_t)row * (size_t)a.ldzg + c;
        if (a.grad) store_row8<DT, PASSING>(a.z_grad, at, z1, valid);
        if (a.grad && a.gated) store_row8<DT, PASSING>(a.z_grad, at + a.cols, z2, valid);
        if (a.y) store_row8<DT, PASSING>(a.y, (size_t)row * (size_t)a.ldy + c, y, valid);
    }
}

namespace {

// Workgroups of 256 threads, or of 64 where those would leave compute units idle.
void shape(int64_t units, dim3& grid, dim3& block) {
    const int threads = units * 16 >= 256 * 1024 ? 256 : 64;
    const int64_t n = (units + threads / 16 - 1) / (threads / 16);
    block = dim3((unsigned)threads);
    grid = dim3((unsigned)(n < (1 << 23) ? n : (1 << 23)));
}

}  // namespace

int launch_activation(const ActArgs& a, int dtype, hipStream_t s) {
    const bool split = a.gated && a.cols % 128 != 0 && a.codes.q != nullptr;
    const int zcols = a.gated ? 2 * a.cols : a.cols;
    const int per = pieces<128>(a.cols) + (split ? pieces<128>(zcols) : 0);
    const int64_t units = (int64_t)a.rows * per;
    dim3 grid, block;
    shape(units, grid, block);
#define DG_ACT(DT, PASSING)                                                                                   \
    return split ? launch_status(activation_forward<DT, true, PASSING>, grid, block, s, a, units, per)        \
                 : launch_status(activation_forward<DT, false, PASSING>, grid, block, s, a, units, per)
#define DG_ACT_DT(DT)              \
    if (a.passing) DG_ACT(DT, true); \
    DG_ACT(DT, false)
    if (dtype == DT_F32) { DG_ACT_DT(DT_F32); }
    if (dtype == DT_F16) { DG_ACT_DT(DT_F16); }
    DG_ACT_DT(DT_BF16);
#undef DG_ACT_DT
#undef DG_ACT
}

int launch_activation_backward(const ActArgs& a, int dtype, hipStream_t s) {
    const int per = pieces<128>(a.cols);
    const int64_t units = (int64_t)a.rows * per;
    dim3 grid, block;
    shape(units, grid, block);
#define DG_ACT(DT)                                                                                  \
    return a.passing ? launch_status(activation_backward<DT, true>, grid, block, s, a, units, per) \
                     : launch_status(activation_backward<DT, false>, grid, block, s, a, units, per)
    if (dtype == DT_F32) DG_ACT(DT_F32);
    if (dtype == DT_F16) DG_ACT(DT_F16);
    DG_ACT(DT_BF16);
#undef DG_ACT
}

}  // namespace dg
