// moe_route.cu -- routing of tokens to experts, and its gradient (sm_100a).
//
// For a token's logits l[0..E): scores p = softmax(l) or sigmoid(l); candidates
// c = p + bias (l itself without a bias: both score functions are monotone, and the
// logits do not tie where saturated scores would); with groups, only the candidates of
// the top_groups groups with the largest sum of their group_top best ones; the k largest
// candidates, ties to the lower index.  Weights from p, see include/mxq.h.
//
// The choice is that of the formula in 64 bits.  The kernel computes p and c in 32 bits
// with a known error and compares: where two candidates that the order depends on lie closer
// than that error allows, the few candidates in question are computed again in 64 bits; where
// two groups at the border do, the whole row is.  With scores spread as a router's are, that
// happens in 0.2% of the rows, so the 64-bit part costs nothing on average.
//
// One warp per row.  Lane l holds the NI consecutive elements l NI .. l NI + NI - 1 (NI the
// power of two that covers E), so that the lowest index of equal candidates is the lowest
// lane's, a group is a run of lanes, and a row loads in 16-byte pieces.  Bound by
// instruction issue: a row of 256 in 8 groups with a bias takes about 750 warp instructions
// (65536 rows: 59 us, 1.2 TB/s), a row of 128 without either about 500.

#include <algorithm>
#include <type_traits>

#include "dependent.cuh"
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
__device__ __forceinline__ void warp_argmax(double& v, int& idx) {
#pragma unroll
    for (int s = 16; s; s >>= 1) {
        const double ov = __shfl_xor_sync(FULL_MASK, v, s);
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
    int gs, gl_log;  // experts of a group; log2 of its lanes where a group is a run of whole lanes, else -1
    bool aligned;    // the row arrays start on 16-byte boundaries
};

// Scores of the lane's elements in 64 bits (softmax over the whole row, or sigmoid); masked
// (-inf) and absent elements get 0.
template <int NI>
__device__ __forceinline__ void scores_in_64(const float (&l)[NI], int score, double (&p)[NI]) {
    if (score == 1) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            double q;
            sigmoid_pair<double>((double)l[i], p[i], q);
            if (l[i] == neg_inf<float>()) p[i] = 0.0;
        }
        return;
    }
    float m = neg_inf<float>();
#pragma unroll
    for (int i = 0; i < NI; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        p[i] = l[i] == neg_inf<float>() ? 0.0 : exp((double)l[i] - (double)m);
        sum += p[i];
    }
    sum = warp_sum(sum);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int i = 0; i < NI; ++i) p[i] *= inv;
}

// How far the 32-bit value of a candidate c = p + b may be from the exact one.
// A softmax score's relative error: l - max rounded (|l - max| 2^-24 <= 104 * 2^-24 before the
// score is zero in 32 bits), exp within 2 units in the last place, the sum of up to 1024 terms
// in chains of 32 + 5 additions, two roundings more: together under 2^-16.
// A sigmoid's: u = __expf(-|l|) is within 2 + 1.173 |l| units in the last place, 124 at
// |l| = 104, with an addition, a reciprocal and a product more under 2^-16 relative; since
// dp = p (1 - p) du / u, and p (1 - p) (2 + 1.173 |l|) < 0.65, under 2^-21 absolute.
// Then the addition's rounding, and the underflow of scores below 2^-126.
constexpr float RT_REL = 0x1p-16f, RT_ABS_SIGMOID = 0x1p-21f;
__device__ __forceinline__ float cand_err(int score, float p, float c) {
    // p comes as c - b, itself rounded
    return (score == 1 ? RT_ABS_SIGMOID : p * RT_REL) + fabsf(c) * 0x1p-22f + 0x1p-126f;
}
// The largest of any score: scores are at most 1.
__device__ __forceinline__ float score_err(int score) { return score == 1 ? RT_ABS_SIGMOID : RT_REL; }

// The choice in 64 bits: lane j < k gets the id of the j-th (-1 if there are fewer).  The
// lane holds the elements lane + 32 i; `sc` is the warp's shared row of E values.
template <int NI>
__device__ __forceinline__ void choose_in_64(const float (&l)[NI], const RouteArgs& a, double* sc, int lane, int& id) {
    const double NEG = neg_inf<double>();
    const bool have_bias = a.bias != nullptr;
    const bool by_p = a.n_groups > 1 && !have_bias && a.group_top == 2;
    double c[NI], p[NI];
    scores_in_64<NI>(l, a.score, p);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        c[i] = l[i] == neg_inf<float>() ? NEG : have_bias ? p[i] + (double)__ldg(a.bias + e) : (double)l[i];
    }
    if (a.n_groups > 1) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) sc[e] = by_p && c[i] != NEG ? p[i] : c[i];
        }
        __syncwarp();
        const int gs = a.gs;
        double best = NEG, second = NEG;
        if (lane < a.n_groups)
            for (int j = 0; j < gs; ++j) {
                const double v = sc[lane * gs + j];
                if (v > best) {
                    second = best;
                    best = v;
                } else if (v > second) {
                    second = v;
                }
            }
        __syncwarp();
        const bool some = best > NEG;
        double gsum = best;
        if (a.group_top == 2 && some && second > NEG) gsum = best + second;
        int before = 0;
        for (int h = 0; h < a.n_groups; ++h) {
            const double o = __shfl_sync(FULL_MASK, gsum, h);
            if (o > gsum || (o == gsum && h < lane)) ++before;
        }
        const unsigned kept = __ballot_sync(FULL_MASK, lane < a.n_groups && some && before < a.top_groups);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (!((kept >> (e < a.E ? e / gs : 0)) & 1u)) c[i] = NEG;
        }
    }
    id = -1;
    for (int j = 0; j < a.k; ++j) {
        double v = NEG;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (c[i] > v) {
                v = c[i];
                at = lane + 32 * i;
            }
        warp_argmax(v, at);
        if (!(v > NEG)) break;
        if (lane == j) id = at;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (at == lane + 32 * i) c[i] = NEG;
    }
}

// ---- 32-bit choice -------------------------------------------------------------------------------

__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
    return r;
}

// The same, NaN if any is.
__device__ __forceinline__ float redux_max_nan(float v) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 1 / v for 1 <= v <= 2, within one unit in the last place.
__device__ __forceinline__ float rcp1(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float widen(float v) { return v; }

// The lane's elements as fp32, -inf past the row.  `vec`: rows and lanes start on the
// boundaries that the widest load wants.
template <int NI, typename L>
__device__ __forceinline__ void load_row(const L* __restrict__ row, int E, bool vec, int lane, float (&l)[NI]) {
    constexpr int BYTES = NI * (int)sizeof(L) < 16 ? NI * (int)sizeof(L) : 16;
    constexpr int PER = BYTES / (int)sizeof(L);  // elements per piece
    const int e0 = lane * NI;
    if (vec && PER > 1) {
#pragma unroll
        for (int i = 0; i < NI; i += PER) {
            L v[PER];
            if (e0 + i < E) {
                if (BYTES == 16)
                    *reinterpret_cast<uint4*>(v) = ld_nc_v4(row + e0 + i);
                else if (BYTES == 8)
                    *reinterpret_cast<uint2*>(v) = ld_nc_v2(row + e0 + i);
                else
                    *reinterpret_cast<uint32_t*>(v) = __ldg(reinterpret_cast<const uint32_t*>(row + e0 + i));
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) l[i + j] = e0 + i < E ? widen(v[j]) : neg_inf<float>();
        }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) l[i] = e0 + i < E ? ld_logit(row + e0 + i) : neg_inf<float>();
    }
}

// Whether load_row may use its pieces: every row starts on a piece's boundary.
template <int NI, typename L>
__host__ __device__ constexpr bool row_vec(int E) {
    return E % (NI * (int)sizeof(L) < 16 ? NI : 16 / (int)sizeof(L)) == 0;
}

// Descending order within the lane, equal values by index: neighbours are exchanged only
// where the later one is larger.
template <int NI>
__device__ __forceinline__ void sort_lane(float (&c)[NI], int (&x)[NI]) {
#pragma unroll
    for (int n = 1; n < NI; ++n)
#pragma unroll
        for (int i = n; i > 0; --i) {
            const bool up = c[i] > c[i - 1];
            const float hi = up ? c[i] : c[i - 1], lo = up ? c[i - 1] : c[i];
            const int xh = up ? x[i] : x[i - 1], xl = up ? x[i - 1] : x[i];
            c[i - 1] = hi, c[i] = lo, x[i - 1] = xh, x[i] = xl;
        }
}

// The row's n best candidates in order, equal ones by index: lane j < 32 gets the j-th
// (id -1 if there is none); the last one asked for also goes to every lane.  Destroys c.
template <int NI>
__device__ __forceinline__ void extract(float (&c)[NI], int n, int lane, int& id, float& val, int& last_id,
                                        float& last_val) {
    constexpr bool SORTED = NI <= 8;  // above, a sort costs more than looking again
    int x[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) x[i] = lane * NI + i;
    if (SORTED) sort_lane<NI>(c, x);
    id = -1;
    val = neg_inf<float>();
    for (int j = 0; j < n; ++j) {
        float head = c[0];
        int at = x[0];
        if (!SORTED) {
#pragma unroll
            for (int i = 1; i < NI; ++i)
                if (c[i] > head) {
                    head = c[i];
                    at = x[i];
                }
        }
        const float m = redux_max(head);
        const unsigned who = __ballot_sync(FULL_MASK, head == m);
        const int win = __ffs(who) - 1;
        const int e = m > neg_inf<float>() ? __shfl_sync(FULL_MASK, at, win) : -1;
        if (lane == j) {
            id = e;
            val = m;
        }
        last_id = e;
        last_val = m;
        if (e < 0) break;  // nothing is left: the same for the ones not asked
        if (lane == win) {
            if (SORTED) {
#pragma unroll
                for (int i = 0; i + 1 < NI; ++i) {
                    c[i] = c[i + 1];
                    x[i] = x[i + 1];
                }
                c[NI - 1] = neg_inf<float>();
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (x[i] == e) c[i] = neg_inf<float>();
            }
        }
    }
}

// The exact value of candidate e, in 64 bits: score + bias (max and sum: softmax's, over the
// row in 64 bits).
__device__ __forceinline__ double exact_candidate(float l, float b, int score, double max, double sum) {
    double p, q;
    if (score == 1)
        sigmoid_pair<double>((double)l, p, q);
    else
        p = exp((double)l - max) / sum;
    return p + (double)b;
}

// Softmax's sum over the row in 64 bits, to every lane.
template <typename L>
__device__ __noinline__ double exact_sum(const L* row, int E, double max, int lane) {
    double s = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) s += exp((double)ld_logit(row + e) - max);
    return warp_sum(s);
}

// The k <= 16 best by a threshold.  The k-th largest of the lanes' own maxima is at most the
// row's k-th best candidate, so the candidates from it up (`slack` lower, where a candidate
// may be that far from its exact value) are all that can be chosen: about -32 ln(1 - k / 32)
// of them for values in no order (9 for k = 8, 22 for k = 16).  They are gathered in index
// order, and each counts the ones before it.  With a bias, candidates closer together than
// their errors are counted again by their values in 64 bits.  Lane j < k gets the j-th id.
// False, with nothing done, where more than 32 are left (rows of equal logits).
struct __align__(16) Picked {
    float val[36];  // 32, and one for what is not picked
    float err[36];
    int id[36];
};
// 1 if the value o of a candidate before (`earlier`) or after this one goes before v.
__device__ __forceinline__ int before(float o, float v, bool earlier) { return o > v || (o == v && earlier); }

template <int NI, typename L>
__device__ __forceinline__ bool select_few(const float (&c)[NI], const RouteArgs& a, bool have_bias, int score,
                                           const L* row, float slack, float top, int lane, Picked* s, int& id) {
    const float NEG = neg_inf<float>();
    float h = c[0];
#pragma unroll
    for (int i = 1; i < NI; ++i) h = fmaxf(h, c[i]);
    float t = NEG;
    for (int j = 0; j < a.k; ++j) {  // equal maxima leave together: the threshold only gets lower
        t = redux_max(h);
        if (h == t) h = NEG;
    }
    // fewer lanes than k have any: all finite ones
    const float low = t > NEG ? fmaxf(t - slack, -3.402823466e38f) : -3.402823466e38f;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) mine += c[i] >= low;
    int pos = mine;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
        const int o = __shfl_up_sync(FULL_MASK, pos, sh);
        if (lane >= sh) pos += o;
    }
    const int cnt = __shfl_sync(FULL_MASK, pos, 31);
    if (cnt > 32) return false;
    pos -= mine;
#pragma unroll
    for (int i = 0; i < NI; ++i) {  // without branches: the others go to a place of their own
        const bool in = c[i] >= low;
        const int at = in ? pos : 32;
        s->val[at] = c[i];
        s->id[at] = lane * NI + i;
        pos += in;
    }
    __syncwarp();
    float v = NEG, err = 0.0f, b = 0.0f;
    int e = -1, rank = 0;
    if (lane < cnt) {
        v = s->val[lane];
        e = s->id[lane];
    }
    if (have_bias) {
        if (lane < cnt) {
            b = __ldg(a.bias + e);
            err = cand_err(score, fabsf(v - b), v);
        }
        s->val[lane] = v;  // the places behind the last hold -inf
        s->err[lane] = err;
        __syncwarp();
        int near = 0;  // candidates that this one may tie with, itself among them
        for (int j = 0; j < cnt; j += 4) {
            const float4 o = *reinterpret_cast<const float4*>(s->val + j);
            const float4 f = *reinterpret_cast<const float4*>(s->err + j);
            rank += before(o.x, v, j < lane) + before(o.y, v, j + 1 < lane) + before(o.z, v, j + 2 < lane) +
                    before(o.w, v, j + 3 < lane);
            // (not of equal infinite ones, which tie by index: their difference is no number)
            near += (fabsf(o.x - v) <= err + f.x) + (fabsf(o.y - v) <= err + f.y) + (fabsf(o.z - v) <= err + f.z) +
                    (fabsf(o.w - v) <= err + f.w);
        }
        if (__any_sync(FULL_MASK, near > 1)) {
            const double sum = score == 0 ? exact_sum<L>(row, a.E, (double)top, lane) : 1.0;
            const double x = lane < cnt ? exact_candidate(ld_logit(row + e), b, score, (double)top, sum) : 0.0;
            rank = 0;
            for (int j = 0; j < cnt; ++j) {
                const double o = __shfl_sync(FULL_MASK, x, j);
                rank += o > x || (o == x && j < lane);
            }
        }
    } else {
        s->val[lane] = v;
        __syncwarp();
        for (int j = 0; j < cnt; j += 4) {
            const float4 o = *reinterpret_cast<const float4*>(s->val + j);
            rank += before(o.x, v, j < lane) + before(o.y, v, j + 1 < lane) + before(o.z, v, j + 2 < lane) +
                    before(o.w, v, j + 3 < lane);
        }
    }
    __syncwarp();
    if (lane < cnt) s->id[rank] = e;
    __syncwarp();
    id = lane < min(cnt, a.k) ? s->id[lane] : -1;
    __syncwarp();
    return true;
}

// The exact choice of one row (rare).
template <int NI, typename L>
__device__ __noinline__ int choose_exact(const L* row, RouteArgs a, double* sc, int lane) {
    float l[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < a.E ? ld_logit(row + e) + 0.0f : neg_inf<float>();
    }
    int id;
    choose_in_64<NI>(l, a, sc, lane, id);
    return id;
}

// MODE: what is known when the kernel is compiled, which frees registers and a quarter of the
// instructions (65536 x 256 in 8 groups: 59 us against 77).  Everything else takes ROUTE_ANY:
// softmax with a bias, groups without one, groups that are not runs of whole lanes, and rows of
// more than 256, for which the modes have not been tried (65536 rows, fp32, with sigmoid and
// bias / in 8 groups too / softmax without a bias: 384 experts 133 / 291 / 79 us, 512 experts
// 149 / 172 / 79, 1024 experts 474 / 524 / 189; 256 by their modes 45 / 57 / 31).
enum { ROUTE_ANY = 0, ROUTE_SIGMOID_BIAS_GROUPS = 1, ROUTE_SIGMOID_BIAS = 2, ROUTE_PLAIN = 3 };
template <int NI, typename L, int MODE>
__global__ void __launch_bounds__(32 * RT_WARPS, NI <= 8 ? 4 : NI <= 16 ? 2 : 1)
    moe_route_kernel(const L* __restrict__ logits, RouteArgs a, float* __restrict__ weights,
                     int32_t* __restrict__ ids) {
    extern __shared__ double route_rows[];
    __shared__ Picked picked[RT_WARPS];
    grid_wait();
    const float NEG = neg_inf<float>(), INF = __int_as_float(0x7F800000);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n_warps = (int64_t)gridDim.x * RT_WARPS;
    const bool vec = a.aligned && row_vec<NI, L>(a.E);
    const bool have_bias = MODE == ROUTE_ANY ? a.bias != nullptr : MODE != ROUTE_PLAIN;
    const bool grouped = MODE == ROUTE_ANY ? a.n_groups > 1 : MODE == ROUTE_SIGMOID_BIAS_GROUPS;
    const int score = MODE == ROUTE_SIGMOID_BIAS_GROUPS || MODE == ROUTE_SIGMOID_BIAS ? 1 : a.score;
    const bool by_p = grouped && !have_bias && a.group_top == 2;  // groups by scores, candidates logits
    const bool need_p = have_bias || by_p;
    const int gs = a.gs, gl_log = a.gl_log, gl = 1 << (gl_log < 0 ? 0 : gl_log);
    const bool runs = MODE == ROUTE_SIGMOID_BIAS_GROUPS || gl_log >= 0;
    float* row_s = reinterpret_cast<float*>(route_rows + (int64_t)warp * a.E);
    constexpr bool KEEP_BIAS = NI <= 8;  // the lane's biases stay in registers
    float bias[KEEP_BIAS ? NI : 1];
    if (KEEP_BIAS)
#pragma unroll
        for (int i = 0; i < NI; ++i) bias[i] = have_bias && lane * NI + i < a.E ? __ldg(a.bias + lane * NI + i) : 0.0f;
    // the largest finite bias, for the roundings of the candidates
    float bias_mag = 0.0f;
    if (have_bias) {
        for (int e = lane; e < a.E; e += 32) {
            const float b = fabsf(__ldg(a.bias + e));
            if (b < INF) bias_mag = fmaxf(bias_mag, b);
        }
        bias_mag = redux_max(bias_mag);
    }
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < a.T; t += n_warps) {
        const L* row = logits + t * a.E;
        float l[NI], c[NI];
        load_row<NI, L>(row, a.E, vec, lane, l);
        float top = l[0], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            top = max_nan(top, l[i]);
            c[i] = l[i];
        }
        top = redux_max_nan(top);
        const bool softmax_sum = score == 0 && (need_p || !a.renorm);
        if (need_p || softmax_sum) {
            float p[NI];
            if (score == 1) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const float u = __expf(-fabsf(l[i])), inv = rcp1(1.0f + u);
                    p[i] = l[i] < 0.0f ? u * inv : inv;  // 0 for -inf
                }
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    p[i] = l[i] == NEG ? 0.0f : expf(l[i] - top);
                    sum += p[i];
                }
                sum = warp_sum(sum);
                if (need_p) {
                    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
                    for (int i = 0; i < NI; ++i) p[i] *= inv;
                }
            }
            if (have_bias) {
                float worst = NEG;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int e = lane * NI + i;
                    const float b = KEEP_BIAS ? bias[KEEP_BIAS ? i : 0] : e < a.E ? __ldg(a.bias + e) : 0.0f;
                    c[i] = l[i] == NEG ? NEG : p[i] + b;
                    worst = max_nan(worst, c[i]);
                }
                if (__any_sync(FULL_MASK, isnan(worst))) top = worst = __int_as_float(0x7FC00000);
            } else if (by_p) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (l[i] != NEG) c[i] = p[i];  // for the groups; the logits come back below
            }
        }
        if (isnan(top) || (score == 0 && top == INF)) {
            if (lane < a.k) {
                weights[t * a.k + lane] = __int_as_float(0x7FC00000);
                ids[t * a.k + lane] = lane;
            }
            continue;
        }
        bool sure = true;
        if (grouped) {
            float best = NEG, second = NEG;
            bool kept;
            int g0;  // the lane's group (the first one where a lane holds several)
            if (runs) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    second = fmaxf(second, fminf(best, c[i]));
                    best = fmaxf(best, c[i]);
                }
                for (int sh = 1; sh < gl; sh <<= 1) {
                    const float ob = __shfl_xor_sync(FULL_MASK, best, sh), os = __shfl_xor_sync(FULL_MASK, second, sh);
                    second = fmaxf(fmaxf(second, os), fminf(best, ob));
                    best = fmaxf(best, ob);
                }
                g0 = lane >> gl_log;
            } else {
                // any other shape: lane g scans group g in shared memory
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (lane * NI + i < a.E) row_s[lane * NI + i] = c[i];
                __syncwarp();
                if (lane < a.n_groups)
                    for (int j = 0; j < gs; ++j) {
                        const float v = row_s[lane * gs + j];
                        second = fmaxf(second, fminf(best, v));
                        best = fmaxf(best, v);
                    }
                __syncwarp();
                g0 = lane;
            }
            const bool some = g0 < a.n_groups && best > NEG;
            float gsum = NEG;
            if (some) gsum = a.group_top == 2 && second > NEG ? best + second : best;
            // the best group at a time, equal ones in order; every lane of a group has its sum
            float h = gsum, lo = NEG;
            kept = false;
            for (int j = 0; j < a.top_groups; ++j) {
                const float m = redux_max(h);
                if (!(m > NEG)) break;
                lo = m;
                const int win = __ffs(__ballot_sync(FULL_MASK, h == m)) - 1;
                if (g0 == (runs ? win >> gl_log : win)) {
                    kept = true;
                    h = NEG;
                }
            }
            if (need_p) {
                // the border: the worst kept group against the best one left out.  Each sum has
                // at most two candidates' errors and one addition's; with a bias the scores are
                // bounded by 1 and the roundings by the candidates' magnitudes
                const float hi = redux_max(h);
                if (hi > NEG) {
                    const float err = by_p ? (lo + hi) * (2.0f * RT_REL) + 0x1p-120f
                                           : 4.0f * score_err(score) + (bias_mag + 1.0f) * 0x1p-19f;
                    sure = lo - hi > err;  // false where both are infinite
                }
            }
            if (runs) {
#pragma unroll
                for (int i = 0; i < NI; ++i) c[i] = !kept ? NEG : by_p ? l[i] : c[i];
            } else {
                const unsigned mask = __ballot_sync(FULL_MASK, kept);
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int e = lane * NI + i;
                    if (by_p) c[i] = l[i];
                    if (e >= a.E || !((mask >> (e / gs)) & 1u)) c[i] = NEG;
                }
            }
        }
        int id = -1;
        if (sure) {
            // no finite candidate is further than half of this from its exact value
            const float slack = have_bias ? 2.0f * score_err(score) + (bias_mag + 1.0f) * 0x1p-20f : 0.0f;
            if (a.k > 16 || !select_few<NI, L>(c, a, have_bias, score, row, slack, top, lane, &picked[warp], id)) {
                // with a bias one more than k, to see that the order is beyond doubt
                int last_id = -1;
                float val = NEG, last_val = NEG;
                extract<NI>(c, have_bias ? a.k + 1 : a.k, lane, id, val, last_id, last_val);
                if (lane >= a.k) id = -1;
                if (have_bias) {
                    // each against the next one (lane j has the j-th, every lane the last), all
                    // with the error of the row's largest score: any candidate further down is
                    // then further away than its own error, too
                    const float pmax = score == 1 ? 1.0f : 1.0f / sum;
                    int nid = __shfl_down_sync(FULL_MASK, id, 1);
                    float nv = __shfl_down_sync(FULL_MASK, val, 1);
                    if (lane == a.k - 1) {
                        nid = last_id;
                        nv = last_val;
                    }
                    const float err = 2.0f * cand_err(score, pmax, bias_mag + 1.0f);
                    const bool close = id >= 0 && nid >= 0 && !(val - nv > err) &&
                                       fabsf(val) < INF;  // infinite candidates tie by index, exactly
                    sure = !__any_sync(FULL_MASK, close);
                }
            }
        }
        if (!sure) id = choose_exact<NI, L>(row, a, route_rows + (int64_t)warp * a.E, lane);
        // ---- weights: lane j < k has the j-th choice
        const bool mine = lane < a.k && id >= 0;
        const float lj = mine ? ld_logit(row + id) : NEG;
        float w = 0.0f;
        if (score == 1) {
            const float u = expf(-fabsf(lj)), inv = rcp1(1.0f + u);
            w = !mine ? 0.0f : lj < 0.0f ? u * inv : inv;
            if (a.renorm) w = __fdividef(w, warp_sum(w) + 1e-20f);
        } else if (a.renorm) {
            const float m = redux_max(lj);
            w = mine ? expf(lj - m) : 0.0f;
            const float s = warp_sum(w);
            w = mine ? __fdividef(w, s) : 0.0f;
        } else {
            w = mine ? __fdividef(expf(lj - top), sum) : 0.0f;
        }
        if (lane < a.k) {
            weights[t * a.k + lane] = w * a.scale;
            ids[t * a.k + lane] = mine ? id : -1;
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
// The lane's NI consecutive values to the row, in the pieces of load_row.
template <int NI>
__device__ __forceinline__ void store_row(float* row, int E, bool vec, int lane, const float (&v)[NI]) {
    const int e0 = lane * NI;
    if (vec && NI >= 2) {
        constexpr int PER = NI < 4 ? 2 : 4;
#pragma unroll
        for (int i = 0; i < NI; i += PER)
            if (e0 + i < E) {
                if (PER == 4)
                    *reinterpret_cast<float4*>(row + e0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                else
                    *reinterpret_cast<float2*>(row + e0 + i) = make_float2(v[i], v[i + 1]);
            }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (e0 + i < E) row[e0 + i] = v[i];
    }
}
template <int NI>
__device__ __forceinline__ void store_row(uint16_t* row, int E, bool vec, int lane, const float (&v)[NI]) {
    const int e0 = lane * NI;
    if (vec && NI >= 2) {
        constexpr int PER = NI < 8 ? (NI < 2 ? 2 : NI) : 8;
#pragma unroll
        for (int i = 0; i < NI; i += PER)
            if (e0 + i < E) {
                uint32_t w[PER > 1 ? PER / 2 : 1];
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) w[j] = cvt_bf16x2(v[i + 2 * j], v[i + 2 * j + 1]);
                if (PER == 8)
                    *reinterpret_cast<uint4*>(row + e0 + i) = *reinterpret_cast<uint4*>(w);
                else if (PER == 4)
                    *reinterpret_cast<uint2*>(row + e0 + i) = *reinterpret_cast<uint2*>(w);
                else
                    *reinterpret_cast<uint32_t*>(row + e0 + i) = w[0];
            }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (e0 + i < E) row[e0 + i] = (uint16_t)cvt_bf16x2(v[i], 0.0f);
    }
}

// sum over the k slots m of r_m (g_j - g_m), for the lane's own slot j: what is left of
// g_j - sum_m g_m r_m without its cancellation where one r_m is near 1 (the r_m sum to 1, up to
// a part that the caller adds).  `pairs`: the warp's room for 32.
__device__ __forceinline__ float pair_sum(float r, float g, int k, int lane, float2* pairs) {
    pairs[lane] = make_float2(r, g);
    __syncwarp();
    float d = 0.0f;
    for (int m = 0; m < k; ++m) {
        const float2 o = pairs[m];
        d = fmaf(o.x, g - o.y, d);
    }
    __syncwarp();
    return d;
}

template <int NI, typename L>
__global__ void __launch_bounds__(32 * RT_WARPS) moe_route_backward_kernel(
    const L* __restrict__ logits, RouteArgs a, const int32_t* __restrict__ ids, const float* __restrict__ gw,
    L* __restrict__ gl) {
    // a row per warp: the lanes' values lie with a stride of NI + 1, so that they meet in
    // different banks
    __shared__ float grad_rows[RT_WARPS][32 * (NI + 1)];
    __shared__ float2 pairs_s[RT_WARPS][32];
    grid_wait();
    const float NEG = neg_inf<float>();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* row_s = grad_rows[warp];
    float2* pairs = pairs_s[warp];
    const bool vec = a.aligned && row_vec<NI, L>(a.E);
    const int64_t n_warps = (int64_t)gridDim.x * RT_WARPS;
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < a.T; t += n_warps) {
        const L* row = logits + t * a.E;
        int id = -1;
        float g = 0.0f;
        if (lane < a.k) {
            id = __ldg(ids + t * a.k + lane);
            if (id < 0 || id >= a.E) id = -1;
            if (id >= 0) g = __ldg(gw + t * a.k + lane) * a.scale;
        }
        const bool mine = id >= 0;
        const float lj = mine ? ld_logit(row + id) : NEG;
        // the chosen entries are marked with their slots' numbers, which also shows whether an
        // index comes twice
        const int at = mine ? id / NI * (NI + 1) + id % NI : 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) row_s[lane * (NI + 1) + i] = 0.0f;
        __syncwarp();
        if (mine) row_s[at] = (float)(lane + 1);
        __syncwarp();
        const bool twice = __any_sync(FULL_MASK, mine && row_s[at] != (float)(lane + 1));
        float d = 0.0f;     // the slot's part of its expert's gradient ...
        bool whole = false;  // ... or all of it
        float base[NI];
        if (a.score == 0 && !a.renorm) {
            load_row<NI, L>(row, a.E, vec, lane, base);
            float m = NEG, s = 0.0f, others = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) m = fmaxf(m, base[i]);
            m = redux_max(m);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                base[i] = base[i] == NEG ? 0.0f : expf(base[i] - m);
                s += base[i];
                others += row_s[lane * (NI + 1) + i] == 0.0f ? base[i] : 0.0f;
            }
            s = warp_sum(s);
            others = warp_sum(others);
            const float inv = s != 0.0f ? 1.0f / s : 0.0f;
            const float p = mine && lj != NEG ? expf(lj - m) * inv : 0.0f;
            d = g * p;
            const float f = -warp_sum(d) * inv;
            if (!twice) {  // p (g - sum_j g_j p_j), the unchosen scores' sum taken as it is
                d = p * fmaf(g, others * inv, pair_sum(p, g, a.k, lane, pairs));
                whole = true;
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) base[i] *= f;
        } else {
#pragma unroll
            for (int i = 0; i < NI; ++i) base[i] = 0.0f;
            if (a.score == 1) {
                float p, q;
                sigmoid_pair<float>(lj, p, q);
                if (!mine) p = 0.0f;
                if (a.renorm) {
                    const float inv = 1.0f / (warp_sum(p) + 1e-20f), r = p * inv;
                    // The constant's own part of the formula, g r q 1e-20 / S; where it is under
                    // 2^-53 of g r q it is taken as 0.  That is far below fp32's rounding of a
                    // sum over pairs; where that sum is empty (k = 1) the gradient is then 0.
                    const float rest = 1e-20f * inv > 0x1p-53f ? 1e-20f * inv : 0.0f;
                    d = r * q * fmaf(g, rest, pair_sum(r, g, a.k, lane, pairs));
                } else {
                    d = g * p * q;
                }
            } else {
                const float m = warp_max(lj);
                const float ex = mine && lj > NEG ? expf(lj - m) : (lj == lj ? 0.0f : lj);
                const float s = warp_sum(ex);
                const float r = mine && s != 0.0f ? ex / s : 0.0f;
                d = r * pair_sum(r, g, a.k, lane, pairs);
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NI; ++i) row_s[lane * (NI + 1) + i] = base[i];
        __syncwarp();
        // the chosen entries; an index that comes twice is added in the order of its slots
        if (twice) {
            for (int j = 0; j < a.k; ++j) {
                if (lane == j && mine) row_s[at] += d;
                __syncwarp();
            }
        } else if (mine) {
            row_s[at] = whole ? d : row_s[at] + d;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NI; ++i) base[i] = row_s[lane * (NI + 1) + i];
        store_row<NI>(gl + t * a.E, a.E, vec, lane, base);
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

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Several CTAs' rows per resident CTA, so that rows of unlike cost even out.
static unsigned route_grid(int64_t T) {
    return (unsigned)std::min<int64_t>((T + RT_WARPS - 1) / RT_WARPS, (int64_t)sm_count() * 16);
}

cudaError_t launch_moe_route(const void* logits, bool bf16, int64_t T, int E, const float* bias, int score,
                             int n_groups, int top_groups, int group_top, int k, bool renorm, float scale,
                             float* weights, int32_t* ids, cudaStream_t stream) {
    RouteArgs a{bias, T, E, k, n_groups, top_groups, group_top, score, renorm ? 1 : 0, scale, E / n_groups, -1,
                aligned16(logits)};
    const size_t smem = n_groups > 1 ? (size_t)RT_WARPS * E * sizeof(double) : 0;  // a row per warp, for the groups
    constexpr int MAX_SMEM = RT_WARPS * 1024 * (int)sizeof(double);                // at the largest E
    return by_width(E, [&](auto ni) {
        constexpr int NI = decltype(ni)::value;
        for (int log = 0; log < 6; ++log)
            if (a.gs == NI << log) a.gl_log = log;
        auto go = [&](auto kernel, auto l) {
            // Without this opt-in the static memory counts within the 48 KB, too.  It stays with the
            // kernel, and other host threads launch it: always the same value, never a call's own.
            if (smem + sizeof(Picked) * RT_WARPS > 47 * 1024) {
                const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
                if (e != cudaSuccess) return e;
            }
            return launch_dependent(kernel, route_grid(T), 32 * RT_WARPS, smem, stream, l, a, weights, ids);
        };
        auto typed = [&](auto mode) {
            constexpr int MODE = decltype(mode)::value;
            return bf16 ? go(moe_route_kernel<NI, uint16_t, MODE>, static_cast<const uint16_t*>(logits))
                        : go(moe_route_kernel<NI, float, MODE>, static_cast<const float*>(logits));
        };
        if constexpr (NI <= 8) {
            if (bias && score == 1 && n_groups > 1 && a.gl_log >= 0)
                return typed(std::integral_constant<int, ROUTE_SIGMOID_BIAS_GROUPS>());
            if (bias && score == 1 && n_groups == 1) return typed(std::integral_constant<int, ROUTE_SIGMOID_BIAS>());
            if (!bias && n_groups == 1) return typed(std::integral_constant<int, ROUTE_PLAIN>());
        }
        return typed(std::integral_constant<int, ROUTE_ANY>());
    });
}

cudaError_t launch_moe_route_backward(const void* logits, bool bf16, int64_t T, int E, const int32_t* ids, int k,
                                      const float* grad_weights, int score, bool renorm, float scale,
                                      void* grad_logits, cudaStream_t stream) {
    const RouteArgs a{nullptr, T, E, k, 1, 1, 1, score, renorm ? 1 : 0, scale, E, -1,
                      aligned16(logits) && aligned16(grad_logits)};
    return by_width(E, [&](auto ni) {
        constexpr int NI = decltype(ni)::value;
        return bf16 ? launch_dependent(moe_route_backward_kernel<NI, uint16_t>, route_grid(T), 32 * RT_WARPS, 0, stream,
                                       static_cast<const uint16_t*>(logits), a, ids, grad_weights,
                                       static_cast<uint16_t*>(grad_logits))
                    : launch_dependent(moe_route_backward_kernel<NI, float>, route_grid(T), 32 * RT_WARPS, 0, stream,
                                       static_cast<const float*>(logits), a, ids, grad_weights,
                                       static_cast<float*>(grad_logits));
    });
}

}  // namespace mxq
