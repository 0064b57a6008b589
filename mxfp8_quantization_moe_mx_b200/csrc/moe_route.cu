// moe_route.cu -- routing of tokens to experts, and its gradient (sm_100a).
//
// For a token's logits l[0..E): scores p = softmax(l) or sigmoid(l); candidates
// c = p + bias (l itself without a bias: both score functions are monotone, and the
// logits do not tie where saturated scores would); with groups, only the candidates of
// the top_groups groups with the largest sum of their group_top best ones; the k largest
// candidates, ties to the lower index.  Weights from p, see include/mxq.h.
//
// The choice is that of the formula in 64 bits.  The kernel computes p and c in 32 bits
// with a known error and compares: where two candidates (or two groups at the border)
// that the order depends on lie closer than that error allows, and are not the same
// logit and the same bias, the row's scores are computed again in 64 bits and the choice
// repeated.  With scores spread as a router's are, that happens in well under one row of
// a hundred, so the 64-bit pass costs nothing on average.
//
// One warp per row, lane l holding the elements l, l + 32, ...; nothing is bound by
// arithmetic throughput, see the launcher for what was measured.

#include <algorithm>
#include <type_traits>

#include "mxq_device.cuh"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int RT_WARPS = 8;

__device__ __forceinline__ float ld_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld_logit(const uint16_t* p) {
    return __uint_as_float((uint32_t)__ldg(p) << 16);
}

__device__ __forceinline__ float exp_(float x) { return expf(x); }
__device__ __forceinline__ double exp_(double x) { return exp(x); }

template <typename R>
__device__ __forceinline__ R neg_inf();
template <>
__device__ __forceinline__ float neg_inf<float>() { return __int_as_float(0xFF800000); }
template <>
__device__ __forceinline__ double neg_inf<double>() { return __longlong_as_double(0xFFF0000000000000ll); }

// sigmoid(l) and 1 - sigmoid(l), both without cancellation
template <typename R>
__device__ __forceinline__ void sigmoid_pair(R l, R& p, R& q) {
    const R t = exp_(-(l < 0 ? -l : l));
    const R inv = (R)1 / ((R)1 + t);
    p = l < 0 ? t * inv : inv;
    q = l < 0 ? inv : t * inv;
}

template <typename R>
__device__ __forceinline__ R warp_max(R v) {
#pragma unroll
    for (int s = 16; s; s >>= 1) {
        const R o = __shfl_xor_sync(FULL_MASK, v, s);
        v = o > v ? o : v;
    }
    return v;
}

template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(FULL_MASK, v, s);
    return v;
}

// The warp's largest (value, lowest index on ties); returned to every lane.
template <typename R>
__device__ __forceinline__ void warp_argmax(R& v, int& idx) {
#pragma unroll
    for (int s = 16; s; s >>= 1) {
        const R ov = __shfl_xor_sync(FULL_MASK, v, s);
        const int oi = __shfl_xor_sync(FULL_MASK, idx, s);
        if (ov > v || (ov == v && oi < idx)) {
            v = ov;
            idx = oi;
        }
    }
}

struct RouteArgs {
    const float* bias;
    int64_t T;
    int E, k, n_groups, top_groups, group_top, score, renorm;
    float scale;
};

// Scores of the lane's elements (softmax over the whole row, or sigmoid); masked (-inf)
// and absent elements get 0.
template <int NI, typename R>
__device__ __forceinline__ void scores(const float (&l)[NI], int score, R (&p)[NI]) {
    if (score == 1) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            R q;
            sigmoid_pair<R>((R)l[i], p[i], q);
            if (l[i] == neg_inf<float>()) p[i] = (R)0;
        }
        return;
    }
    float m = neg_inf<float>();
#pragma unroll
    for (int i = 0; i < NI; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    R sum = (R)0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        p[i] = l[i] == neg_inf<float>() ? (R)0 : exp_((R)l[i] - (R)m);
        sum += p[i];
    }
    sum = warp_sum(sum);
    const R inv = sum > (R)0 ? (R)1 / sum : (R)0;
#pragma unroll
    for (int i = 0; i < NI; ++i) p[i] *= inv;
}

// How far the 32-bit value of a candidate c = p + b may be from the exact one: the score's
// relative error (l - max rounded: |l - max| 2^-24 <= 104 * 2^-24 before the score is zero
// in 32 bits; exp within 2 units in the last place; the sum of up to 1024 terms in chains
// of 32 + 5 additions; two roundings more: together under 2^-16), the addition's rounding,
// and the underflow of scores below 2^-126.
constexpr float RT_REL = 0x1p-16f;
__device__ __forceinline__ float cand_err(float p, float c) {
    return p * RT_REL + fabsf(c) * 0x1p-23f + 0x1p-126f;
}

// The choice, in type R.  On return lane j < k holds the id of the j-th choice in `id` (-1
// if there are fewer candidates).  Returns false (float only) if the order is in doubt.
// `sc` is the warp's shared row of E values of type R.
template <int NI, typename R>
__device__ __forceinline__ bool choose(const float (&l)[NI], const RouteArgs& a, R* sc, int lane, int& id) {
    const R NEG = neg_inf<R>();
    const bool have_bias = a.bias != nullptr;
    const bool need_p = have_bias || (a.n_groups > 1 && a.group_top == 2);
    R c[NI];
    R p[NI];
    if (need_p) scores<NI, R>(l, a.score, p);
    bool sure = true;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        if (!need_p) p[i] = (R)0;
        if (l[i] == neg_inf<float>())
            c[i] = NEG;
        else if (have_bias)
            c[i] = p[i] + (R)__ldg(a.bias + e);
        else
            c[i] = (R)l[i];
    }
    if (a.n_groups > 1) {
        // the value that groups are ranked by: the candidate, or the score where the sum of
        // two is wanted and the candidates are logits
        const bool by_p = !have_bias && a.group_top == 2;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) sc[e] = by_p && c[i] != NEG ? p[i] : c[i];
        }
        __syncwarp();
        const int gs = a.E / a.n_groups;
        R best = NEG, second = NEG;
        if (lane < a.n_groups) {
            for (int j = 0; j < gs; ++j) {
                // start at the lane's own number so that the lanes meet in different banks
                int jj = j + lane;
                if (jj >= gs) jj -= gs * (jj / gs);
                const R v = sc[lane * gs + jj];
                if (v > best) {
                    second = best;
                    best = v;
                } else if (v > second) {
                    second = v;
                }
            }
        }
        __syncwarp();
        const bool some = best > NEG;
        R gsum = best;
        if (a.group_top == 2 && some && second > NEG) gsum = best + second;
        int before = 0;
        for (int h = 0; h < a.n_groups; ++h) {
            const R o = __shfl_sync(FULL_MASK, gsum, h);
            if (o > gsum || (o == gsum && h < lane)) ++before;
        }
        const bool kept = lane < a.n_groups && some && before < a.top_groups;
        const unsigned kept_mask = __ballot_sync(FULL_MASK, kept);
        if (sizeof(R) == 4 && need_p) {
            // the border: the worst kept group against the best one left out
            float lo = warp_max(kept ? -(float)gsum : neg_inf<float>());
            float hi = warp_max(lane < a.n_groups && some && !kept ? (float)gsum : neg_inf<float>());
            // each group's sum has at most two candidates' errors and one addition's; with a
            // bias the scores are bounded by 1 and the roundings by the candidates' magnitudes
            const float mag = warp_max(some ? fabsf((float)best) + (second > NEG ? fabsf((float)second) : 0.0f) : 0.0f);
            if (hi > neg_inf<float>() && lo > neg_inf<float>()) {
                lo = -lo;
                const float err = by_p ? (lo + hi) * (2.0f * RT_REL) + 0x1p-120f : 4.0f * RT_REL + mag * 0x1p-21f;
                if (!(lo - hi > err)) sure = false;
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            const int g = e < a.E ? e / gs : 0;
            if (!((kept_mask >> g) & 1u)) c[i] = NEG;
        }
    }
    // k extractions (one more where the order may be in doubt); a lane keeps its own best
    id = -1;
    const bool check = sizeof(R) == 4 && have_bias;
    const int n = check ? a.k + 1 : a.k;
    R prev = NEG;
    float prev_l = 0.0f, prev_b = 0.0f, prev_err = 0.0f;
    for (int j = 0; j < n; ++j) {
        R v = NEG;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (c[i] > v) {
                v = c[i];
                at = lane + 32 * i;
            }
        warp_argmax(v, at);
        if (!(v > NEG)) break;
        if (j < a.k && lane == j) id = at;
        float wl = 0.0f, wp = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (at == lane + 32 * i) {
                c[i] = NEG;
                wl = l[i];
                wp = (float)p[i];
            }
        if (check) {
            wl = __shfl_sync(FULL_MASK, wl, at & 31);
            wp = __shfl_sync(FULL_MASK, wp, at & 31);
            const float wb = __ldg(a.bias + at);
            const float err = cand_err(wp, (float)v);
            // infinite candidates (an infinite bias) tie by index, exactly
            if (j > 0 && !((float)(prev - v) > prev_err + err) && !(wl == prev_l && wb == prev_b) &&
                fabsf((float)v) < __int_as_float(0x7F800000))
                sure = false;
            prev = v;
            prev_l = wl;
            prev_b = wb;
            prev_err = err;
        }
    }
    return sizeof(R) == 8 || sure;
}

template <int NI, typename L>
__global__ void __launch_bounds__(32 * RT_WARPS) moe_route_kernel(const L* __restrict__ logits, RouteArgs a,
                                                                  float* __restrict__ weights,
                                                                  int32_t* __restrict__ ids) {
    extern __shared__ double route_rows[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double* row_s = route_rows + (int64_t)warp * a.E;
    const int64_t n_warps = (int64_t)gridDim.x * RT_WARPS;
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < a.T; t += n_warps) {
        const L* row = logits + t * a.E;
        float l[NI];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            l[i] = neg_inf<float>();
            if (e < a.E) {
                l[i] = ld_logit(row + e) + 0.0f;  // -0 becomes +0: the two are equal
                // a NaN, or what makes one of a candidate, spoils the row
                bad |= isnan(l[i]) || (a.score == 0 && l[i] == __int_as_float(0x7F800000));
                if (a.bias) bad |= isnan(__ldg(a.bias + e)) && l[i] != neg_inf<float>();
            }
        }
        if (__any_sync(FULL_MASK, bad)) {
            if (lane < a.k) {
                weights[t * a.k + lane] = __int_as_float(0x7FC00000);
                ids[t * a.k + lane] = lane;
            }
            continue;
        }
        int id;
        if (!choose<NI, float>(l, a, reinterpret_cast<float*>(row_s), lane, id))
            choose<NI, double>(l, a, row_s, lane, id);
        // ---- weights: lane j < k has the j-th choice
        const bool mine = lane < a.k && id >= 0;
        const float lj = mine ? ld_logit(row + id) + 0.0f : neg_inf<float>();
        float w = 0.0f;
        if (a.score == 1) {
            float q;
            sigmoid_pair<float>(lj, w, q);
            if (!mine) w = 0.0f;
            if (a.renorm) w = w / (warp_sum(w) + 1e-20f);
        } else if (a.renorm) {
            const float m = warp_max(lj);
            w = mine ? expf(lj - m) : 0.0f;
            const float s = warp_sum(w);
            w = mine ? w / s : 0.0f;
        } else {
            float m = neg_inf<float>(), s = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) m = fmaxf(m, l[i]);
            m = warp_max(m);
#pragma unroll
            for (int i = 0; i < NI; ++i) s += l[i] == neg_inf<float>() ? 0.0f : expf(l[i] - m);
            s = warp_sum(s);
            w = mine ? expf(lj - m) / s : 0.0f;
        }
        if (lane < a.k) {
            weights[t * a.k + lane] = w * a.scale;
            ids[t * a.k + lane] = id;
        }
    }
}

// ---- gradient of the logits -------------------------------------------------------------------
//
// With s the scale, g_j the gradients of the weights and p_j the chosen scores:
//   softmax             dl_e = p_e (s g_e [e chosen] - s sum_j g_j p_j)
//   softmax, renorm     r_j = softmax of the chosen logits: dl_j = s r_j (g_j - sum_m g_m r_m)
//   sigmoid             dl_j = s g_j p_j (1 - p_j)
//   sigmoid, renorm     r_j = p_j / (sum p + 1e-20): dl_j = s r_j (1 - p_j) (g_j - sum_m g_m r_m)
// and 0 for every other expert.  A warp per row builds the row in shared memory (scattered
// entries) and writes it out in order.
template <typename L>
__device__ __forceinline__ void st_grad(L* p, float v);
template <>
__device__ __forceinline__ void st_grad<float>(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void st_grad<uint16_t>(uint16_t* p, float v) { *p = (uint16_t)cvt_bf16x2(v, 0.0f); }

template <int NI, typename L>
__global__ void __launch_bounds__(32 * RT_WARPS) moe_route_backward_kernel(
    const L* __restrict__ logits, RouteArgs a, const int32_t* __restrict__ ids, const float* __restrict__ gw,
    L* __restrict__ gl) {
    extern __shared__ float grad_rows[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* row_s = grad_rows + (int64_t)warp * a.E;
    const int64_t n_warps = (int64_t)gridDim.x * RT_WARPS;
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < a.T; t += n_warps) {
        const L* row = logits + t * a.E;
        int id = -1;
        float g = 0.0f;
        if (lane < a.k) {
            id = ids[t * a.k + lane];
            if (id < 0 || id >= a.E) id = -1;
            if (id >= 0) g = gw[t * a.k + lane] * a.scale;
        }
        const bool mine = id >= 0;
        const float lj = mine ? ld_logit(row + id) : neg_inf<float>();
        float d = 0.0f, dot = 0.0f;
        float base[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) base[i] = 0.0f;
        if (a.score == 1) {
            float p, q;
            sigmoid_pair<float>(lj, p, q);
            if (!mine) p = 0.0f;
            if (a.renorm) {
                const float r = p / (warp_sum(p) + 1e-20f);
                d = r * q * (g - warp_sum(g * r));
            } else {
                d = g * p * q;
            }
        } else if (a.renorm) {
            const float m = warp_max(lj);
            const float ex = mine && lj > neg_inf<float>() ? expf(lj - m) : (lj == lj ? 0.0f : lj);
            const float s = warp_sum(ex);
            const float r = mine && s != 0.0f ? ex / s : 0.0f;
            d = r * (g - warp_sum(g * r));
        } else {
            float m = neg_inf<float>(), s = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane + 32 * i;
                base[i] = e < a.E ? ld_logit(row + e) : neg_inf<float>();
                m = fmaxf(m, base[i]);
            }
            m = warp_max(m);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                base[i] = base[i] == neg_inf<float>() ? 0.0f : expf(base[i] - m);
                s += base[i];
            }
            s = warp_sum(s);
            const float inv = s != 0.0f ? 1.0f / s : 0.0f;
            const float p = mine && lj != neg_inf<float>() ? expf(lj - m) * inv : 0.0f;
            d = g * p;
            dot = warp_sum(d);
#pragma unroll
            for (int i = 0; i < NI; ++i) base[i] *= -dot * inv;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) row_s[e] = base[i];
        }
        __syncwarp();
        // the chosen entries; an index that comes twice is added in the order of its slots
        const unsigned same = __match_any_sync(FULL_MASK, mine ? id : -1 - lane);
        if (__any_sync(FULL_MASK, (same & (same - 1)) != 0)) {
            for (int j = 0; j < a.k; ++j) {
                if (lane == j && mine) row_s[id] += d;
                __syncwarp();
            }
        } else if (mine) {
            row_s[id] += d;
        }
        __syncwarp();
        L* out = gl + t * a.E;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) st_grad<L>(out + e, row_s[e]);
        }
        __syncwarp();
    }
}

template <typename F>
cudaError_t by_width(int E, F&& f) {
    const int ni = (E + 31) / 32;
    if (ni <= 1) return f(std::integral_constant<int, 1>());
    if (ni <= 2) return f(std::integral_constant<int, 2>());
    if (ni <= 4) return f(std::integral_constant<int, 4>());
    if (ni <= 8) return f(std::integral_constant<int, 8>());
    if (ni <= 16) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

}  // namespace

cudaError_t launch_moe_route(const void* logits, bool bf16, int64_t T, int E, const float* bias, int score,
                             int n_groups, int top_groups, int group_top, int k, bool renorm, float scale,
                             float* weights, int32_t* ids, cudaStream_t stream) {
    const RouteArgs a{bias, T, E, k, n_groups, top_groups, group_top, score, renorm ? 1 : 0, scale};
    const int64_t ctas = (T + RT_WARPS - 1) / RT_WARPS;
    const unsigned grid = (unsigned)std::min<int64_t>(ctas, (int64_t)sm_count() * 8);
    const size_t smem = n_groups > 1 ? (size_t)RT_WARPS * E * sizeof(double) : 0;
    return by_width(E, [&](auto ni) {
        constexpr int NI = decltype(ni)::value;
        cudaError_t e = cudaSuccess;
        if (bf16) {
            if (smem > 48 * 1024)
                e = cudaFuncSetAttribute(moe_route_kernel<NI, uint16_t>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
            if (e != cudaSuccess) return e;
            moe_route_kernel<NI, uint16_t><<<grid, 32 * RT_WARPS, smem, stream>>>(
                static_cast<const uint16_t*>(logits), a, weights, ids);
        } else {
            if (smem > 48 * 1024)
                e = cudaFuncSetAttribute(moe_route_kernel<NI, float>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
            if (e != cudaSuccess) return e;
            moe_route_kernel<NI, float><<<grid, 32 * RT_WARPS, smem, stream>>>(static_cast<const float*>(logits), a,
                                                                               weights, ids);
        }
        return cudaGetLastError();
    });
}

cudaError_t launch_moe_route_backward(const void* logits, bool bf16, int64_t T, int E, const int32_t* ids, int k,
                                      const float* grad_weights, int score, bool renorm, float scale,
                                      void* grad_logits, cudaStream_t stream) {
    const RouteArgs a{nullptr, T, E, k, 1, 1, 1, score, renorm ? 1 : 0, scale};
    const int64_t ctas = (T + RT_WARPS - 1) / RT_WARPS;
    const unsigned grid = (unsigned)std::min<int64_t>(ctas, (int64_t)sm_count() * 8);
    const size_t smem = (size_t)RT_WARPS * E * sizeof(float);
    return by_width(E, [&](auto ni) {
        constexpr int NI = decltype(ni)::value;
        if (bf16)
            moe_route_backward_kernel<NI, uint16_t><<<grid, 32 * RT_WARPS, smem, stream>>>(
                static_cast<const uint16_t*>(logits), a, ids, grad_weights, static_cast<uint16_t*>(grad_logits));
        else
            moe_route_backward_kernel<NI, float><<<grid, 32 * RT_WARPS, smem, stream>>>(
                static_cast<const float*>(logits), a, ids, grad_weights, static_cast<float*>(grad_logits));
        return cudaGetLastError();
    });
}

}  // namespace mxq
