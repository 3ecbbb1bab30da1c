// route.hip -- the choice of experts for each token, its gradient, and the plan that
// sorts the tokens by expert.
//
// Scores and choice values are fp64: which of two experts is taken can hang on less than
// an fp32 rounding of their scores, and the whole computation is a few tens of fp64
// operations per logit. Choice values become 64-bit whole numbers of the same order (a
// NaN the largest), so that a comparison of (value, index) has no special cases.
#include <algorithm>

#include "device_common.h"
#include "experts.h"
#include "launch.h"

namespace dg {

// The order of doubles as unsigned numbers; 0 is below all of them, -0 counts as 0.
__device__ __forceinline__ uint64_t order_key(double x) {
    if (x != x) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | (1ull << 63);
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

// One wave's scores of a token, lane l holding experts l, l + 64, ...
template <int R, int DT>
__device__ __forceinline__ void token_scores(const RouteArgs& a, int t, int lane, double (&s)[R]) {
    typedef typename Elem<DT>::type T;
    const T* row = static_cast<const T*>(a.logits) + (size_t)t * (size_t)a.ld;
    double x[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int e = lane + 64 * j;
        x[j] = e < a.experts ? (double)decode<DT>(row[e]) : -__builtin_inf();
    }
    if (a.score == GEMM_SCORE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < R; ++j) s[j] = lane + 64 * j < a.experts ? 1.0 / (1.0 + exp(-x[j])) : 0.0;
        return;
    }
    double top = x[0];
#pragma unroll
    for (int j = 1; j < R; ++j) top = x[j] > top || x[j] != x[j] ? x[j] : top;
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const double o = __shfl_xor(top, d);
        top = o > top || o != o ? o : top;
    }
    double total = 0;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        s[j] = lane + 64 * j < a.experts ? exp(x[j] - top) : 0.0;
        total += s[j];
    }
    total = wave_sum(total);
#pragma unroll
    for (int j = 0; j < R; ++j) s[j] = s[j] / total;
}

// One wave per token.
template <int R, int DT>
__global__ __launch_bounds__(256) void route(RouteArgs a) {
    __shared__ double choice[4][R * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t first = (int64_t)blockIdx.x * 4; first < a.tokens; first += (int64_t)gridDim.x * 4) {
        const bool on = first + wave < a.tokens;
        const int t = (int)(on ? first + wave : a.tokens - 1);
        double s[R];
        token_scores<R, DT>(a, t, lane, s);
        uint64_t key[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int e = lane + 64 * j;
            const double c = a.bias && e < a.experts ? s[j] + (double)a.bias[e] : s[j];
            key[j] = e < a.experts ? order_key(c) : 0;
            choice[wave][e] = c;
        }
        if (a.groups > 1) {
            __syncthreads();
            // lane g: the sum of the largest choice values of group g, and g + 64, ...
            const int per = a.experts / a.groups;
            uint64_t best[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int grp = lane + 64 * j;
                best[j] = 0;
                if (grp >= a.groups) continue;
                double v[4];
                uint64_t k[4] = {0, 0, 0, 0};
                for (int i = 0; i < per; ++i) {
                    double cv = choice[wave][grp * per + i];
                    uint64_t ck = order_key(cv);
#pragma unroll
                    for (int q = 0; q < 4; ++q)  // insertion into the four largest
                        if (ck > k[q]) {
                            const double tv = v[q];
                            const uint64_t tk = k[q];
                            v[q] = cv;
                            k[q] = ck;
                            cv = tv;
                            ck = tk;
                        }
                }
                double sum = v[0];
#pragma unroll
                for (int q = 1; q < 4; ++q)
                    if (q < a.group_top) sum += v[q];
                best[j] = order_key(sum);
            }
            uint64_t kept[R];  // bit mask over the groups, 64 at a time
#pragma unroll
            for (int j = 0; j < R; ++j) kept[j] = 0;
            for (int i = 0; i < a.top_groups; ++i) {
                uint64_t k = 0;
                int at = 0;
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (best[j] > k) k = best[j], at = lane + 64 * j;
#pragma unroll
                for (int d = 32; d; d >>= 1) {
                    const uint64_t ok = __shfl_xor((unsigned long long)k, d);
                    const int oa = __shfl_xor(at, d);
                    if (ok > k || (ok == k && oa < at)) k = ok, at = oa;
                }
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    if (at >> 6 == j) kept[j] |= 1ull << (at & 63);
                    if (at == lane + 64 * j) best[j] = 0;
                }
            }
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int e = lane + 64 * j, grp = e / per;
                if (e >= a.experts) continue;
                bool in = false;
#pragma unroll
                for (int q = 0; q < R; ++q)
                    if (grp >> 6 == q) in = (kept[q] >> (grp & 63)) & 1;
                if (!in) key[j] = order_key(-__builtin_inf());
            }
            __syncthreads();
        }
        // lane i keeps pick i
        double mine = 0, total = 0;
        int mine_at = 0;
        for (int i = 0; i < a.top_k; ++i) {
            uint64_t k = 0;
            int at = lane;
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (key[j] > k) k = key[j], at = lane + 64 * j;
#pragma unroll
            for (int d = 32; d; d >>= 1) {
                const uint64_t ok = __shfl_xor((unsigned long long)k, d);
                const int oa = __shfl_xor(at, d);
                if (ok > k || (ok == k && oa < at)) k = ok, at = oa;
            }
            double w = 0;
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (at >> 6 == j) {
                    w = s[j];
                    if (at == lane + 64 * j) key[j] = 0;
                }
            w = __shfl(w, at & 63);
            total += w;
            if (lane == i) mine = w, mine_at = at;
        }
        if (on && lane < a.top_k) {
            const double w = (a.renorm ? mine / total : mine) * (double)a.factor;
            a.index[(size_t)t * a.top_k + lane] = mine_at;
            a.weight[(size_t)t * a.top_k + lane] = (float)w;
        }
    }
}

// With p_j the chosen scores, g_j = factor * dL/dw_j (renorm: g_j = (factor dL/dw_j -
// sum_i factor dL/dw_i p_i / P) / P, P = sum p), the logits' gradient is
//   sigmoid: ds (1 - s) s        softmax: s (ds - sum_e ds_e s_e),   ds_e = sum of g_j at e
template <int R, int DT>
__global__ __launch_bounds__(256) void route_backward(RouteArgs a) {
    typedef typename Elem<DT>::type T;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t first = (int64_t)blockIdx.x * 4 + wave; first < a.tokens; first += (int64_t)gridDim.x * 4) {
        const int t = (int)first;
        double s[R], ds[R];
        token_scores<R, DT>(a, t, lane, s);
        const int at = lane < a.top_k ? a.index_in[(size_t)t * a.top_k + lane] : -1;
        const bool in = at >= 0 && at < a.experts;
        double g = lane < a.top_k ? (double)a.weight_grad[(size_t)t * a.top_k + lane] * (double)a.factor : 0.0;
        if (!in) g = 0;
        if (a.renorm) {
            double p = 0;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const double v = __shfl(s[j], at & 63);
                if (in && at >> 6 == j) p = v;
            }
            const double total = wave_sum(p), dot = wave_sum(g * p);
            g = in ? (g - dot / total) / total : 0;
        }
#pragma unroll
        for (int j = 0; j < R; ++j) ds[j] = 0;
        for (int i = 0; i < a.top_k; ++i) {
            const double gi = __shfl(g, i);
            const int ai = __shfl(in ? at : -1, i);
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (ai == lane + 64 * j) ds[j] += gi;
        }
        double dot = 0;
        if (a.score == GEMM_SCORE_SOFTMAX) {
#pragma unroll
            for (int j = 0; j < R; ++j) dot += ds[j] * s[j];
            dot = wave_sum(dot);
        }
        T* out = static_cast<T*>(a.grad) + (size_t)t * (size_t)a.ldg;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int e = lane + 64 * j;
            if (e >= a.experts) continue;
            const double d = a.score == GEMM_SCORE_SOFTMAX ? s[j] * (ds[j] - dot) : ds[j] * s[j] * (1 - s[j]);
            store_out(out, DT, (size_t)e, (float)d);
        }
    }
}

template <int DT>
int launch_route_dt(const RouteArgs& a, bool backward, hipStream_t s) {
    const dim3 grid((unsigned)std::min((a.tokens + 3) / 4, 1 << 20)), block(256);
    const int r = (a.experts + 63) / 64;
    if (backward) {
        if (r <= 1) return launch_status(route_backward<1, DT>, grid, block, s, a);
        if (r <= 2) return launch_status(route_backward<2, DT>, grid, block, s, a);
        if (r <= 4) return launch_status(route_backward<4, DT>, grid, block, s, a);
        if (r <= 8) return launch_status(route_backward<8, DT>, grid, block, s, a);
        return launch_status(route_backward<16, DT>, grid, block, s, a);
    }
    if (r <= 1) return launch_status(route<1, DT>, grid, block, s, a);
    if (r <= 2) return launch_status(route<2, DT>, grid, block, s, a);
    if (r <= 4) return launch_status(route<4, DT>, grid, block, s, a);
    if (r <= 8) return launch_status(route<8, DT>, grid, block, s, a);
    return launch_status(route<16, DT>, grid, block, s, a);
}

int launch_route(const RouteArgs& a, int dtype, bool backward, hipStream_t s) {
    if (dtype == DT_F32) return launch_route_dt<DT_F32>(a, backward, s);
    if (dtype == DT_F16) return launch_route_dt<DT_F16>(a, backward, s);
    return launch_route_dt<DT_BF16>(a, backward, s);
}

// ---------------------------------------------------------------------------- the plan
// The pairs' ranks within their expert: each wave takes 256 pairs, 64 at a time. The lanes
// with the same expert find each other by comparing its bits (ballots), and a counter for
// each wave and expert carries on from one 64 to the next; no atomics, so the order is
// that of the pairs. Returns a lane's four experts and ranks within its wave.
__device__ __forceinline__ void wave_ranks(const DispatchArgs& a, int chunk, int* counter, int (&ex)[4],
                                           int (&rank)[4]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t i = (int64_t)chunk * kDispatchChunk + wave * 256 + u * 64 + lane;
        const int e = i < a.n ? a.index[i] : -1;
        ex[u] = e >= 0 && e < a.experts ? e : -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int e = ex[u];
        uint64_t same = __ballot(e >= 0);
#pragma unroll
        for (int b = 0; b < 10; ++b) {
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

__global__ __launch_bounds__(256) void dispatch_count(DispatchArgs a) {
    __shared__ int counter[4][kMaxExperts];
    const int tid = threadIdx.x;
    for (int i = tid; i < 4 * kMaxExperts; i += 256) (&counter[0][0])[i] = 0;
    __syncthreads();
    int ex[4], rank[4];
    wave_ranks(a, blockIdx.x, counter[tid >> 6], ex, rank);
    __syncthreads();
    for (int e = tid; e < a.experts; e += 256)
        a.work[(size_t)blockIdx.x * a.experts + e] = counter[0][e] + counter[1][e] + counter[2][e] + counter[3][e];
}

__global__ __launch_bounds__(256) void dispatch_place(DispatchArgs a) {
    __shared__ int counter[4][kMaxExperts];  // then: first row of each wave's pairs of an expert
    __shared__ int start[kMaxExperts + 1], count[kMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < 4 * kMaxExperts; i += 256) (&counter[0][0])[i] = 0;
    __syncthreads();
    int ex[4], rank[4];
    wave_ranks(a, blockIdx.x, counter[wave], ex, rank);
    __syncthreads();
    for (int e = tid; e < a.experts; e += 256) {
        int before = 0, total = 0;
        if (a.chunks > 1) {
            for (int c = 0; c < a.chunks; ++c) {
                const int n = a.work[(size_t)c * a.experts + e];
                before += c < (int)blockIdx.x ? n : 0;
                total += n;
            }
        } else {
            total = counter[0][e] + counter[1][e] + counter[2][e] + counter[3][e];
        }
        count[e] = total;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int n = counter[w][e];
            counter[w][e] = before;
            before += n;
        }
    }
    __syncthreads();
    if (wave == 0) {  // offsets: the padded counts added up, 64 experts at a time
        int64_t base = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 64) {
            const int e = e0 + lane;
            const int64_t n = e < a.experts ? ((int64_t)count[e] + a.align - 1) / a.align * a.align : 0;
            int64_t sum = n;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t v = __shfl_up((long long)sum, d);
                if (lane >= d) sum += v;
            }
            if (e < a.experts) start[e] = (int)(base + sum - n);
            base += __shfl((long long)sum, 63);
        }
        if (lane == 0) start[a.experts] = (int)base;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t i = (int64_t)blockIdx.x * kDispatchChunk + wave * 256 + u * 64 + lane;
        if (i >= a.n) continue;
        const int e = ex[u];
        const int p = e >= 0 ? start[e] + counter[wave][e] + rank[u] : -1;
        a.position[i] = p;
        if (p >= 0 && p < a.capacity) a.rows[p] = (int)(i / a.top_k);
    }
    // padding
    const int step = gridDim.x;
    for (int e = blockIdx.x; e < a.experts; e += step)
        for (int p = start[e] + count[e] + tid; p < start[e + 1]; p += 256) a.rows[p] = -1;
    for (int64_t p = (int64_t)start[a.experts] + (int64_t)blockIdx.x * 256 + tid; p < a.capacity; p += (int64_t)step * 256)
        a.rows[p] = -1;
    if (blockIdx.x == 0) {
        for (int e = tid; e <= a.experts; e += 256) a.offsets[e] = start[e];
        for (int e = tid; e < a.experts; e += 256) a.counts[e] = count[e];
    }
}

int launch_dispatch(const DispatchArgs& a, hipStream_t s) {
    if (a.chunks > 1) {
        const int rc = launch_status(dispatch_count, dim3((unsigned)a.chunks), dim3(256), s, a);
        if (rc) return rc;
    }
    return launch_status(dispatch_place, dim3((unsigned)a.chunks), dim3(256), s, a);
}

}  // namespace dg
