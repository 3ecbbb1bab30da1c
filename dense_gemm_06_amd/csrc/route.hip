// route.hip -- the choice of experts for each token, its gradient, and the plan that
// sorts the tokens by expert.
//
// Scores and choice values are fp64: which of two experts is taken can hang on less than
// an fp32 rounding of their scores. The work is bound by instruction issue, not by memory
// (16384 tokens x 256 experts: 16 MB of logits, 4 us), so a token gets as few lanes as hold
// its experts 16 to a lane: four tokens of up to 256 experts share a wave, and what is
// done once for a token (the reductions, the picks) is done for four at a time. A lane's
// experts are neighbours, so the lowest lane that holds a maximum holds its lowest index.
#include <algorithm>

#include "device_common.h"
#include "experts.h"
#include "extents.h"
#include "launch.h"

namespace dg {

// e^x in fp64 for -708 <= x <= 708 (a NaN stays one): Cody-Waite reduction by multiples of
// ln 2 (the high part of 33 bits, so that k * high is exact), a Taylor polynomial on
// |r| <= 0.35 (the first term left out is below 5e-18), and k added to the exponent. k is
// rounded by adding 1.5 * 2^52, which leaves it in the low bits: about half the instructions
// of the library's exp, whose special cases are not needed here.
// The coefficients stay in scalar registers, where one operand of an fma may come from:
// left to itself the compiler copies each into a vector register first.
struct ExpTerms {
    double c[11], hi, lo, inv, magic;
    __device__ __forceinline__ ExpTerms() {
        const double f[11] = {1.0 / 6227020800.0, 1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0,
                              1.0 / 362880.0,     1.0 / 40320.0,     1.0 / 5040.0,     1.0 / 720.0,
                              1.0 / 120.0,        1.0 / 24.0,        1.0 / 6.0};
#pragma unroll
        for (int i = 0; i < 11; ++i) {
            c[i] = f[i];
            asm("" : "+s"(c[i]));
        }
        hi = -0x1.62e42feep-1;
        lo = -0x1.a39ef35793c76p-33;
        inv = 1.4426950408889634;
        magic = 6755399441055744.0;
        asm("" : "+s"(hi), "+s"(lo), "+s"(inv), "+s"(magic));
    }
};

__device__ __forceinline__ double exp64(const ExpTerms& x, double v) {
    const double kd = fma(v, x.inv, x.magic), k = kd - x.magic;
    double r = fma(k, x.hi, v);
    r = fma(k, x.lo, r);
    double p = fma(x.c[0], r, x.c[1]);
#pragma unroll
    for (int i = 2; i < 11; ++i) p = fma(p, r, x.c[i]);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    const uint64_t u = (uint64_t)__double_as_longlong(p);
    const uint32_t up = (uint32_t)(u >> 32) + ((uint32_t)__double_as_longlong(kd) << 20);
    return __longlong_as_double((long long)(((uint64_t)up << 32) | (uint32_t)u));
}

// 1 / d for normal d >= 1 (a NaN stays one): the hardware estimate, two Newton steps and one
// of the residual.
__device__ __forceinline__ double rcp64(double d) {
    double r = __builtin_amdgcn_rcp(d);
    r = fma(fma(-d, r, 1.0), r, r);
    r = fma(fma(-d, r, 1.0), r, r);
    return fma(fma(-d, r, 1.0), r, r);
}

// e^(x - m), m >= x, and the sigmoid of an fp32 number, 0 below e^-708 (fp64's normal numbers
// end there). x - m is exact in fp64 where it counts, and its NaNs (infinities) stay.
__device__ __forceinline__ double exp_shifted(const ExpTerms& c, float x, float m) {
    const float d = x - m;  // only to compare
    const double e = exp64(c, d < -708.0f ? -708.0 : (double)x - (double)m);
    return d < -708.0f ? 0.0 : e;
}
__device__ __forceinline__ double sigmoid_of(const ExpTerms& c, float x) {
    const float y = x < -708.0f ? -708.0f : x > 708.0f ? 708.0f : x;
    const double s = rcp64(1.0 + exp64(c, -(double)y));
    return x < -708.0f ? 0.0 : s;
}

// Value of the lane that differs in the bits of D (1, 2, 4 mirrored, 8 mirrored, 16, 32).
template <int D>
__device__ __forceinline__ int lane_swap(int x) {
    if constexpr (D == 1) return __builtin_amdgcn_update_dpp(0, x, 0xB1, 0xF, 0xF, true);        // quad_perm 1,0,3,2
    else if constexpr (D == 2) return __builtin_amdgcn_update_dpp(0, x, 0x4E, 0xF, 0xF, true);   // quad_perm 2,3,0,1
    else if constexpr (D == 4) return __builtin_amdgcn_update_dpp(0, x, 0x141, 0xF, 0xF, true);  // mirror of 8
    else if constexpr (D == 8) return __builtin_amdgcn_update_dpp(0, x, 0x140, 0xF, 0xF, true);  // mirror of 16
    else return __shfl_xor(x, D);
}
template <int D>
__device__ __forceinline__ double lane_swap(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = (uint32_t)lane_swap<D>((int)(uint32_t)u), hi = (uint32_t)lane_swap<D>((int)(uint32_t)(u >> 32));
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// Reductions over each W lanes (a power of two), with the result in all of them. The mirrors
// of 8 and 16 do as well as exchanges once the lanes of a quad (of 8) agree.
template <int W, int D = 1, typename F>
__device__ __forceinline__ double lanes_reduce(double x, F f) {
    if constexpr (D < W) return lanes_reduce<W, D * 2>(f(x, lane_swap<D>(x)), f);
    else return x;
}
template <int W>
__device__ __forceinline__ double lanes_max(double x) {
    return lanes_reduce<W>(x, [](double a, double b) { return __builtin_fmax(a, b); });
}
template <int W>
__device__ __forceinline__ double lanes_sum(double x) {
    return lanes_reduce<W>(x, [](double a, double b) { return a + b; });
}

template <int W, int D = 1>
__device__ __forceinline__ float lanes_maxf(float x) {
    if constexpr (D < W)
        return lanes_maxf<W, D * 2>(fmaxf(x, __uint_as_float((uint32_t)lane_swap<D>((int)__float_as_uint(x)))));
    else return x;
}

// A choice value as a number that compares like it under max: NaN is the largest.
constexpr double kAbsent = -__builtin_inf();  // below every key
__device__ __forceinline__ double order_key(double x) {
    const double top = 1.7976931348623157e308;
    return x != x ? __builtin_inf() : __builtin_fmin(__builtin_fmax(x, -top), top);
}

// The key of a group: the sum of its largest values' keys, `top` the largest of them and `low`
// the smallest. NaN where top is one, or where infinities of both signs meet.
__device__ __forceinline__ double group_key(double sum, double top, double low) {
    const double most = 1.7976931348623157e308;  // infinity's key
    const bool nan = top == __builtin_inf() || (top == most && low == -most);
    return nan ? __builtin_inf() : order_key(sum);
}

// The largest of each W lanes' keys, and where: the lane within the W and the register.
// Ties go to the lowest lane, then the lowest register.
template <int W, int R>
__device__ __forceinline__ double lanes_argmax(const double (&key)[R], int lane, int& at_lane, int& at_reg) {
    double top = key[0];
#pragma unroll
    for (int j = 1; j < R; ++j) top = __builtin_fmax(top, key[j]);
    const double best = lanes_max<W>(top);
    uint64_t hit = __ballot(top == best);
    if constexpr (W < 64) hit = (hit >> (lane & ~(W - 1))) & ((1ull << W) - 1);
    at_lane = __builtin_ctzll(hit);
    at_reg = 0;
#pragma unroll
    for (int j = R - 1; j >= 0; --j)
        if (key[j] == best) at_reg = j;
    return best;
}

// A token's scores, W lanes to a token, lane l of them holding experts l*R .. l*R + R-1.
template <int W, int R, int DT>
__device__ __forceinline__ void token_scores(const RouteArgs& a, const ExpTerms& c, int t, int l, double (&s)[R]) {
    typedef typename Elem<DT>::type T;
    const T* row = static_cast<const T*>(a.logits) + (size_t)t * (size_t)a.ld + l * R;
    const int left = a.experts - l * R;
    T raw[R];
    if (left >= R) {
        __builtin_memcpy(raw, row, sizeof raw);
    } else {
#pragma unroll
        for (int j = 0; j < R; ++j) raw[j] = j < left ? row[j] : T(0);
    }
    float x[R];
#pragma unroll
    for (int j = 0; j < R; ++j) x[j] = j < left ? decode<DT>(raw[j]) : -__builtin_inff();
    if (a.score == GEMM_SCORE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            s[j] = sigmoid_of(c, x[j]);  // 0 for the absent -inf
            if ((j & 3) == 3) __builtin_amdgcn_sched_barrier(0);  // four at a time: enough in flight, fewer registers
        }
        return;
    }
    float top = x[0];
#pragma unroll
    for (int j = 1; j < R; ++j) top = fmaxf(top, x[j]);
    const float m = lanes_maxf<W>(top);  // NaNs show in the sum
    double total = 0;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        s[j] = exp_shifted(c, x[j], m);
        total += s[j];
        if ((j & 3) == 3) __builtin_amdgcn_sched_barrier(0);
    }
    const double inv = rcp64(lanes_sum<W>(total));
#pragma unroll
    for (int j = 0; j < R; ++j) s[j] *= inv;
}

// 64 / W tokens to a wave, four waves to a workgroup. The scores wait in LDS; the picks
// go by the choice values rounded to fp32 (16 registers, one instruction a comparison, where
// fp64 takes three times as many): rounding keeps their order but for ties, and where any
// token's largest is not alone the wave decides by the fp64 values. NaN (which max and == pass
// over) stands for what is picked, masked by the groups or does not exist: -inf would tie with
// an expert that a bias of -inf excludes.
// ANY_GROUPS: groups that cut lanes, or more than the two largest of a group (a kernel of its
// own, for the others' registers).
// 16384 tokens x 256 experts, sigmoid, 8 groups: 100 us with a wave to a token and fp64
// picks, 32 us with 16 lanes to a token, 27 us with fp32 picks, 22 us with 123 registers. Half
// of its cycles issue the 2000 vector instructions of each wave (four tokens; four waves to a
// SIMD, all at once; a fifth in fp64, at the same rate); the rest is the launch and latency: of
// the logits, of LDS, and of the picks, each of which waits for the one before.
template <int W, int R, int DT, bool ANY_GROUPS>
__global__ __launch_bounds__(256) void route(RouteArgs a) {
    constexpr int PER = 64 / W;
    __shared__ double values[4][64 * R];
    __shared__ uint8_t kept[4][64 * R];
    __shared__ uint16_t picks[4][PER * kMaxTopK];
    __shared__ float shift[W * R];  // the bias
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & (W - 1), sub = lane / W;
    double* mine = &values[wave][sub * W * R];
    const int left = a.experts - l * R;
    for (int e = threadIdx.x; e < a.experts; e += 256) shift[e] = a.bias ? a.bias[e] : 0.0f;
    __syncthreads();
    const ExpTerms terms;
    const int64_t step = (int64_t)gridDim.x * 4 * PER;
    for (int64_t first = ((int64_t)blockIdx.x * 4 + wave) * PER; first < a.tokens; first += step) {
        const bool on = first + sub < a.tokens;
        const int t = (int)(on ? first + sub : a.tokens - 1);
        float key[R], bias[R];
#pragma unroll
        for (int j = 0; j < R; ++j) bias[j] = j < left ? shift[l * R + j] : 0.0f;
        double v0 = kAbsent, v1 = kAbsent;  // the lane's two largest choice values
        {
            double s[R];
            token_scores<W, R, DT>(a, terms, t, l, s);
#pragma unroll
            for (int j = 0; j < R; ++j) mine[l * R + j] = s[j];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const double k = j < left ? order_key(s[j] + (double)bias[j]) : kAbsent;
                key[j] = j < left ? (float)k : __builtin_nanf("");
                v1 = __builtin_fmax(v1, __builtin_fmin(v0, k));
                v0 = __builtin_fmax(v0, k);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (a.groups > 1) {
            const int per = a.experts / a.groups;
            if constexpr (!ANY_GROUPS) {
                // a group is group_lanes whole lanes: its two largest by exchanges among them
                auto merge = [&](double o0, double o1) {
                    v1 = __builtin_fmax(__builtin_fmin(v0, o0), v0 > o0 ? v1 : o1);
                    v0 = __builtin_fmax(v0, o0);
                };
                if (a.group_lanes > 1) merge(lane_swap<1>(v0), lane_swap<1>(v1));
                if (a.group_lanes > 2) merge(lane_swap<2>(v0), lane_swap<2>(v1));
                if (a.group_lanes > 4) merge(lane_swap<4>(v0), lane_swap<4>(v1));
                double best[1] = {left > 0 ? group_key(a.group_top == 2 ? v0 + v1 : v0, v0, a.group_top == 2 ? v1 : v0) : kAbsent};
                bool in = false;
                for (int i = 0; i < a.top_groups; ++i) {
                    int at, reg;
                    lanes_argmax<W, 1>(best, lane, at, reg);
                    if ((l ^ at) < a.group_lanes) {  // the winner's lanes
                        in = true;
                        best[0] = kAbsent;
                    }
                }
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (!in) key[j] = __builtin_nanf("");
            } else {
                // any group: lane l sums the largest values of groups l*R .. l*R + R-1
                uint8_t* keep = &kept[wave][sub * W * R];
                double best[R];
#pragma unroll 1
                for (int j = 0; j < R; ++j) {
                    const int grp = l * R + j;
                    double v[4] = {kAbsent, kAbsent, kAbsent, kAbsent};
                    if (grp < a.groups)
#pragma unroll 4
                        for (int i = 0; i < per; ++i) {
                            const int e = grp * per + i;
                            double x = order_key(mine[e] + (double)shift[e]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const double lower = __builtin_fmin(v[q], x);
                                v[q] = __builtin_fmax(v[q], x);
                                x = lower;
                            }
                        }
                    double sum = v[0], low = v[0];
#pragma unroll
                    for (int q = 1; q < 4; ++q)
                        if (q < a.group_top) {
                            sum += v[q];
                            low = v[q];
                        }
                    const double b = grp < a.groups ? group_key(sum, v[0], low) : kAbsent;
#pragma unroll
                    for (int q = 0; q < R; ++q)
                        if (q == j) best[q] = b;
                    keep[grp] = 0;
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                for (int i = 0; i < a.top_groups; ++i) {
                    int at, reg;
                    lanes_argmax<W, R>(best, lane, at, reg);
                    if (l == at) {
#pragma unroll
                        for (int j = 0; j < R; ++j)
                            if (j == reg) best[j] = kAbsent;
                        keep[l * R + reg] = 1;
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (j < left && !keep[(l * R + j) / per]) key[j] = __builtin_nanf("");
            }
        }
        // picks in descending order; lane i of the token keeps pick i (and W + i)
        for (int i = 0; i < a.top_k; ++i) {
            float top = key[0];
#pragma unroll
            for (int j = 1; j < R; ++j) top = fmaxf(top, key[j]);
            const float best = lanes_maxf<W>(top);
            int hits = 0, reg = 0;
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                hits += __popcll(__ballot(key[j] == best));
                if (key[j] == best) reg = j;
            }
            int at;
            if (hits == PER) {  // one for each token
                uint64_t hit = __ballot(top == best);
                if constexpr (W < 64) hit = (hit >> (lane & ~(W - 1))) & ((1ull << W) - 1);
                at = __builtin_ctzll(hit);
            } else {
                double full[R];
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    const int e = l * R + j;
                    full[j] = kAbsent;
                    if (key[j] == best) full[j] = order_key(mine[e] + (double)bias[j]);
                    if ((j & 3) == 3) __builtin_amdgcn_sched_barrier(0);
                }
                lanes_argmax<W, R>(full, lane, at, reg);
            }
            if (l == at) {
                picks[wave][sub * kMaxTopK + i] = (uint16_t)(at * R + reg);
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (j == reg) key[j] = __builtin_nanf("");
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int i0 = l < a.top_k ? picks[wave][sub * kMaxTopK + l] : 0;
        const int i1 = l + W < a.top_k ? picks[wave][sub * kMaxTopK + l + W] : 0;
        const double w0 = l < a.top_k ? mine[i0] : 0.0, w1 = l + W < a.top_k ? mine[i1] : 0.0;
        const double total = lanes_sum<W>(w0 + w1), scale = a.factor;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (!on) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = h * W + l;
            if (i >= a.top_k) continue;
            const double w = h ? w1 : w0;
            a.index[(size_t)t * a.top_k + i] = h ? i1 : i0;
            a.weight[(size_t)t * a.top_k + i] = (float)((a.renorm ? w / total : w) * scale);
        }
    }
}

// With p_j the chosen scores, g_j = factor * dL/dw_j (renorm: g_j = (factor dL/dw_j -
// sum_i factor dL/dw_i p_i / P) / P, P = sum p), the logits' gradient is
//   sigmoid: ds (1 - s) s        softmax: s (ds - sum_e ds_e s_e),   ds_e = sum of g_j at e
// A sigmoid's gradient needs only the chosen scores; a softmax's all of them, and the
// chosen ones are fetched through LDS. ds is laid out over the experts in LDS, one pick of
// each token at a time (a repeated choice adds up in the picks' order). 16384 tokens x 256
// experts, sigmoid: 14 us for the 16 MB of gradient and the chosen logits (4 us of memory);
// latency of the picks' LDS additions, and the launch.
template <int W, int R, int DT>
__global__ __launch_bounds__(256) void route_backward(RouteArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr int PER = 64 / W;
    __shared__ double values[4][64 * R];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & (W - 1), sub = lane / W;
    double* mine = &values[wave][sub * W * R];
    const bool softmax = a.score == GEMM_SCORE_SOFTMAX;
    const ExpTerms terms;
    const int64_t step = (int64_t)gridDim.x * 4 * PER;
    for (int64_t first = ((int64_t)blockIdx.x * 4 + wave) * PER; first < a.tokens; first += step) {
        const bool on = first + sub < a.tokens;
        const int t = (int)(on ? first + sub : a.tokens - 1);
        double s[R];
        if (softmax) {
            token_scores<W, R, DT>(a, terms, t, l, s);
#pragma unroll
            for (int j = 0; j < R; ++j) mine[l * R + j] = s[j];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        int at[2];
        double g[2], p[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = h * W + l;
            at[h] = i < a.top_k ? a.index_in[(size_t)t * a.top_k + i] : -1;
            if (at[h] >= a.experts) at[h] = -1;
            g[h] = p[h] = 0;
            if (at[h] >= 0) {
                g[h] = (double)a.weight_grad[(size_t)t * a.top_k + i] * (double)a.factor;
                if (softmax) p[h] = mine[at[h]];
                else
                    p[h] = sigmoid_of(terms, decode<DT>(static_cast<const T*>(a.logits)[(size_t)t * (size_t)a.ld + at[h]]));
            }
        }
        if (a.renorm) {
            const double total = lanes_sum<W>(p[0] + p[1]), dot = lanes_sum<W>(g[0] * p[0] + g[1] * p[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) g[h] = at[h] >= 0 ? (g[h] - dot / total) / total : 0.0;
        }
        const double dot = softmax ? lanes_sum<W>(g[0] * p[0] + g[1] * p[1]) : 0.0;
        if (!softmax) {
#pragma unroll
            for (int h = 0; h < 2; ++h) g[h] = g[h] * p[h] * (1 - p[h]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int j = 0; j < R; ++j) mine[l * R + j] = 0;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        for (int i = 0; i < a.top_k; ++i) {
            const int x = i < W ? at[0] : at[1];
            if ((i & (W - 1)) == l && x >= 0) mine[x] += i < W ? g[0] : g[1];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        T* out = static_cast<T*>(a.grad) + (size_t)t * (size_t)a.ldg + l * R;
        const int left = on ? a.experts - l * R : 0;
        T raw[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const double ds = mine[l * R + j];
            store_out(raw, DT, j, (float)(softmax ? s[j] * (ds - dot) : ds));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (left >= R) {
            __builtin_memcpy(out, raw, sizeof raw);
        } else {
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (j < left) out[j] = raw[j];
        }
    }
}

// Lanes to a token and experts to a lane: 16 lanes up to 256 experts, 64 above.
template <int W, int R, int DT>
int launch_route_as(RouteArgs a, bool backward, hipStream_t s) {
    const dim3 grid((unsigned)std::min(pieces<4 * (64 / W)>(a.tokens), 1 << 20)), block(256);
    if (backward) return launch_status(route_backward<W, R, DT>, grid, block, s, a);
    // groups that are 1, 2, 4 or 8 whole lanes (of a token's 16)
    const int per = a.experts / a.groups, lanes = per / R;
    a.group_lanes = W == 16 && a.groups > 1 && per % R == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 8 ? lanes : 0;
    if (a.groups > 1 && (a.group_lanes == 0 || a.group_top > 2)) return launch_status(route<W, R, DT, true>, grid, block, s, a);
    return launch_status(route<W, R, DT, false>, grid, block, s, a);
}

template <int DT>
int launch_route_dt(const RouteArgs& a, bool backward, hipStream_t s) {
    if (a.experts <= 16) return launch_route_as<16, 1, DT>(a, backward, s);
    if (a.experts <= 32) return launch_route_as<16, 2, DT>(a, backward, s);
    if (a.experts <= 64) return launch_route_as<16, 4, DT>(a, backward, s);
    if (a.experts <= 128) return launch_route_as<16, 8, DT>(a, backward, s);
    if (a.experts <= 256) return launch_route_as<16, 16, DT>(a, backward, s);
    if (a.experts <= 512) return launch_route_as<64, 8, DT>(a, backward, s);
    return launch_route_as<64, 16, DT>(a, backward, s);
}

int launch_route(const RouteArgs& a, int dtype, bool backward, hipStream_t s) {
    if (dtype == DT_F32) return launch_route_dt<DT_F32>(a, backward, s);
    if (dtype == DT_F16) return launch_route_dt<DT_F16>(a, backward, s);
    return launch_route_dt<DT_BF16>(a, backward, s);
}

// ---------------------------------------------------------------------------- the plan
// The pairs' ranks within their expert: each of the 16 waves takes 256 pairs, 64 at a time.
// The lanes with the same expert find each other by comparing its bits (ballots), and a
// counter for each wave and expert carries on from one 64 to the next; no atomics, so the
// order is that of the pairs. Returns a lane's four experts and ranks within its wave.
// 131072 pairs, 256 experts: 5 us to count, 10 us to place (with chunks of 1024 pairs, whose
// 128 counts each workgroup added up one load at a time, 41 us); a single chunk 5 us.
constexpr int kDispatchWaves = kDispatchChunk / 256;

__device__ __forceinline__ void wave_ranks(const DispatchArgs& a, int chunk, int* counter, int (&ex)[4],
                                           int (&rank)[4]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t i = (int64_t)chunk * kDispatchChunk + wave * 256 + u * 64 + lane;
        const int e = i < a.n ? a.index[i] : -1;
        ex[u] = e >= 0 && e < a.experts ? e : -1;
    }
    const int bits = 32 - __builtin_clz(a.experts);  // wave-uniform; experts >= 1
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int e = ex[u];
        uint64_t same = __ballot(e >= 0);
        for (int b = 0; b < bits; ++b) {
            const uint64_t one = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? one : ~one;
        }
        const int before = e >= 0 ? counter[e] : 0;
        const int below = __popcll(same & ((1ull << lane) - 1));
        rank[u] = before + below;
        // the wave's LDS accesses run in order; the fences keep the compiler from moving them
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (e >= 0 && below == 0) counter[e] = before + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

__global__ __launch_bounds__(1024) void dispatch_count(DispatchArgs a) {
    __shared__ int counter[kDispatchWaves * kMaxExperts];  // [wave][expert]
    const int tid = threadIdx.x, E = a.experts;
    for (int i = tid; i < kDispatchWaves * E; i += 1024) counter[i] = 0;
    __syncthreads();
    int ex[4], rank[4];
    wave_ranks(a, blockIdx.x, counter + (tid >> 6) * E, ex, rank);
    __syncthreads();
    for (int e = tid; e < E; e += 1024) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kDispatchWaves; ++w) n += counter[w * E + e];
        a.work[(size_t)blockIdx.x * E + e] = n;
    }
}

__global__ __launch_bounds__(1024) void dispatch_place(DispatchArgs a) {
    __shared__ int counter[kDispatchWaves * kMaxExperts];  // then: first row of each wave's pairs of an expert
    __shared__ int start[kMaxExperts + 1], count[kMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = a.experts;
    for (int i = tid; i < kDispatchWaves * E; i += 1024) counter[i] = 0;
    __syncthreads();
    int ex[4], rank[4];
    wave_ranks(a, blockIdx.x, counter + wave * E, ex, rank);
    __syncthreads();
    for (int e = tid; e < E; e += 1024) {
        int before = 0, total = 0;
        if (a.chunks > 1) {
            // the chunks' counts, sixteen loads in flight
            for (int c0 = 0; c0 < a.chunks; c0 += 16) {
                int n[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) n[u] = a.work[(size_t)min(c0 + u, a.chunks - 1) * E + e];
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const int c = c0 + u;
                    before += c < (int)blockIdx.x ? n[u] : 0;
                    total += c < a.chunks ? n[u] : 0;
                }
            }
        }
#pragma unroll
        for (int w = 0; w < kDispatchWaves; ++w) {
            const int n = counter[w * E + e];
            counter[w * E + e] = before;
            before += n;
        }
        count[e] = a.chunks > 1 ? total : before;
    }
    __syncthreads();
    if (wave == 0) {  // offsets: the padded counts added up, 64 experts at a time
        int64_t base = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            const int64_t n = e < E ? (int64_t)(((uint32_t)count[e] + (uint32_t)a.align - 1) / (uint32_t)a.align) * a.align : 0;
            int64_t sum = n;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t v = __shfl_up((long long)sum, d);
                if (lane >= d) sum += v;
            }
            if (e < E) start[e] = (int)(base + sum - n);
            base += __shfl((long long)sum, 63);
        }
        if (lane == 0) start[E] = (int)base;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t i = (int64_t)blockIdx.x * kDispatchChunk + wave * 256 + u * 64 + lane;
        if (i >= a.n) continue;
        const int e = ex[u];
        const int p = e >= 0 ? start[e] + counter[wave * E + e] + rank[u] : -1;
        a.position[i] = p;
        if (p >= 0 && p < a.capacity) a.rows[p] = (int)((uint32_t)i / (uint32_t)a.top_k);
    }
    // padding: an expert's by one wave
    const int waves = (int)gridDim.x * kDispatchWaves;
    for (int e = (int)blockIdx.x * kDispatchWaves + wave; e < E; e += waves)
        stride_walk((int64_t)start[e] + count[e] + lane, start[e + 1], 64, [&](int p) { a.rows[p] = -1; });
    stride_walk((int64_t)start[E] + (int64_t)blockIdx.x * 1024 + tid, a.capacity, (int64_t)gridDim.x * 1024,
                [&](int p) { a.rows[p] = -1; });
    if (blockIdx.x == 0) {
        for (int e = tid; e <= E; e += 1024) a.offsets[e] = start[e];
        for (int e = tid; e < E; e += 1024) a.counts[e] = count[e];
    }
}

int launch_dispatch(const DispatchArgs& a, hipStream_t s) {
    if (a.chunks > 1) {
        const int rc = launch_status(dispatch_count, dim3((unsigned)a.chunks), dim3(1024), s, a);
        if (rc) return rc;
    }
    return launch_status(dispatch_place, dim3((unsigned)a.chunks), dim3(1024), s, a);
}

}  // namespace dg
