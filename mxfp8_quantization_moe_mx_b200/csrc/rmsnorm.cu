// rmsnorm.cu -- residual addition, root-mean-square norm and MXFP8 quantization in one
// pass, and the norm's gradient (sm_100a).
//
//   h = bf16(x + residual)            (x itself without a residual)
//   r = 1 / sqrt(mean_d h^2 + eps)    (fp32)
//   y = bf16(h r w)
//   q, s = 1x32 MXFP8 blocks of y     (the bytes mx_quantize gives for y)
//
// Everything is bound by HBM: a row is read once, stays in registers through the two
// reductions (sum of squares over the CTA, block maxima over four lanes) and leaves as codes.
// A warp holds 32 V consecutive 8-element vectors of a row, lane l the vectors l, l + 32, ...,
// so four neighbouring lanes hold one 32-element block and a warp's 8 V scale bytes leave in
// one run.  The sums are fp32: a thread adds at most 32 squares, then 5 shuffle steps and at
// most 32 warps' sums, so the relative error stays under 2^-18.

#include <algorithm>
#include <type_traits>

#include "mxq.h"
#include "dependent.cuh"
#include "mxq_launch.h"

namespace mxq {

namespace {

// Plain (not read-only-path) 16-byte load: the residual stream may be updated in place.
__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// Two fp32 operations at once (sm_100): d = a b + c, a b.
struct f2 {
    float x, y;
};
__device__ __forceinline__ unsigned long long pk(f2 v) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ f2 unpk(unsigned long long v) {
    f2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)), "l"(pk(c)));
    return unpk(r);
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)));
    return unpk(r);
}
__device__ __forceinline__ f2 bf2(uint32_t w) { return {bf16_lo(w), bf16_hi(w)}; }

// The i-th pair of a vector of eight bf16.
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Sums of bf16 pairs, rounded once (the exact sum of two bf16 that an fp32 addition would
// round first is never near a midpoint of bf16, so this is also bf16(fp32 sum)).
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
    return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z), add_bf16x2(a.w, b.w));
}

// Eight consecutive weights as they are stored, and as four pairs of fp32.
template <typename W>
struct W8;
template <>
struct W8<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t* w) { v = __ldg(reinterpret_cast<const uint4*>(w)); }
    __device__ __forceinline__ f2 pair(int j) const { return bf2(word(v, j)); }
};
template <>
struct W8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* w) {
        a = __ldg(reinterpret_cast<const float4*>(w));
        b = __ldg(reinterpret_cast<const float4*>(w) + 1);
    }
    __device__ __forceinline__ f2 pair(int j) const {
        return j == 0 ? f2{a.x, a.y} : j == 1 ? f2{a.z, a.w} : j == 2 ? f2{b.x, b.y} : f2{b.z, b.w};
    }
};
// The thread's i-th vector of its V; `warp`: which of its row's warps the thread's is.
template <int V>
__device__ __forceinline__ int vec_of(int i, int warp) {
    return (warp * V + i) * 32 + (int)(threadIdx.x & 31);
}
template <int V>
__device__ __forceinline__ int vec_of(int i) {
    return vec_of<V>(i, (int)(threadIdx.x >> 5));
}

// Sum over the CTA, returned to every thread.  `part` holds 2 x 32 floats; `turn`
// alternates between calls, so that one barrier a call is enough (none for a single warp,
// unless it is asked for).
__device__ __forceinline__ float cta_sum(float v, float* part, int turn, bool barrier = false) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(FULL_MASK, v, s);
    if (n == 1 && !barrier) return v;
    if (lane == 0) part[32 * turn + warp] = v;
    __syncthreads();
    v = lane < n ? part[32 * turn + lane] : 0.0f;
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(FULL_MASK, v, s);
    return v;
}

// ---- forward -------------------------------------------------------------------------------------

// A block's codes (eight per lane) and its scale, where a block may hold Inf or NaN (SPECIAL)
// or not.
template <bool SPECIAL>
__device__ __forceinline__ uint2 codes8(const uint4& o, uint32_t b) {
    if (SPECIAL && b == 255u) return make_uint2(nan4(o.x, o.y), nan4(o.z, o.w));
    const float mul = mx_mult(b);
    return make_uint2(quant4(o.x, o.y, mul), quant4(o.z, o.w, mul));
}

// One row's norm and codes from its packed sums h[] (V vectors per thread), stored.  `base`:
// the element of the thread's first vector; the others follow 256 elements apart.
template <int V, typename W>
__device__ __forceinline__ void norm_row(const uint4 (&h)[V], const W8<W> (&w)[V], float r, int64_t base, int nv,
                                         int warp, uint16_t* y, uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    const int lane = threadIdx.x & 31;
    uint4 o[V];
    uint32_t am[V], top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        uint32_t p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f2 f = mul2(mul2(bf2(word(h[i], j)), f2{r, r}), w[i].pair(j));
            p[j] = cvt_bf16x2(f.x, f.y);
        }
        o[i] = make_uint4(p[0], p[1], p[2], p[3]);
        uint32_t m = mag2(amax2(amax2(p[0], p[1]), amax2(p[2], p[3])));
        m = max(m & 0xFFFFu, m >> 16);
        m = max(m, __shfl_xor_sync(FULL_MASK, m, 1));
        am[i] = max(m, __shfl_xor_sync(FULL_MASK, m, 2));
        top = max(top, am[i]);
    }
    if (y) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (vec_of<V>(i, warp) < nv) *reinterpret_cast<uint4*>(y + base + 256 * i) = o[i];
    }
    uint32_t mine = 0;  // lane l < 8 V: the scale of the warp's block l
    if (!__any_sync(FULL_MASK, top >= 0x7F80u)) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t b = e8m0_of_finite_amax(am[i]);
            if (vec_of<V>(i, warp) < nv) *reinterpret_cast<uint2*>(q + base + 256 * i) = codes8<false>(o[i], b);
            const uint32_t t = __shfl_sync(FULL_MASK, b, (lane & 7) * 4);
            if ((lane >> 3) == i) mine = t;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t b = e8m0_of_amax(am[i]);
            if (vec_of<V>(i, warp) < nv) *reinterpret_cast<uint2*>(q + base + 256 * i) = codes8<true>(o[i], b);
            const uint32_t t = __shfl_sync(FULL_MASK, b, (lane & 7) * 4);
            if ((lane >> 3) == i) mine = t;
        }
    }
    const int block = warp * 8 * V + lane;
    if (lane < 8 * V && block < nv / 4) s[(base - 8 * vec_of<V>(0, warp)) / 32 + block] = (uint8_t)mine;
}

template <int V>
__device__ __forceinline__ float sum_squares(const uint4 (&h)[V]) {
    f2 sq = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f2 f = bf2(word(h[i], j));
            sq = fma2(f, f, sq);
        }
    return sq.x + sq.y;
}

// V vectors per thread straight from global memory: a row's loads are all in flight at once,
// and enough rows are on an SM to cover the reduction; nothing persists, so a CTA's exit and
// the next one's loads overlap the others' arithmetic.  WARP_ROW: a warp per row (eight to a
// CTA, no barrier), else a CTA per row.  65536 rows with a residual, bf16 weights:
//   D = 5120   four vectors 342 us (6.9 TB/s; the codes of the last rows stay in L2), two 402,
//              one 441; persistent CTAs with a ring of bulk-copied rows 395
//   D = 16384  four 1108, two 1471;  D = 2560  173, 180;  D = 1536  106, 107
//   D = 1024   two 72, a warp per row 79;  D = 512  a warp 39, two 69;  D = 256  21, 68
// fp32 weights take the same forms, though only D = 5120 was measured with them: four vectors
// 404 us.  They need more registers than the 64 that the bound of 1024 threads leaves (88 bytes
// a thread are spilled).  With y and rstd written too: bf16 443, fp32 481.
template <int V, bool WARP_ROW, typename W>
__global__ void __launch_bounds__(WARP_ROW ? 256 : 1024) rmsnorm_mx_kernel(
    const uint16_t* x, const uint16_t* residual, const W* __restrict__ w, int64_t M, int D, float eps,
    uint16_t* res_out, uint16_t* y, uint8_t* __restrict__ q, uint8_t* __restrict__ s, float* __restrict__ rstd) {
    __shared__ float part[64];
    grid_wait();
    const int nv = D / 8;
    const int warp = WARP_ROW ? 0 : (int)(threadIdx.x >> 5);
    const int64_t first = WARP_ROW ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = WARP_ROW ? (int64_t)gridDim.x * 8 : gridDim.x;
    int turn = 0;
    for (int64_t m = first; m < M; m += step, turn ^= 1) {
        const int64_t base = m * D + 8 * vec_of<V>(0, warp);
        uint4 h[V];
        W8<W> g[V] = {};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool in = vec_of<V>(i, warp) < nv;
            h[i] = in ? ld_v4(x + base + 256 * i) : make_uint4(0, 0, 0, 0);
            if (in) g[i].load(w + 8 * vec_of<V>(i, warp));
            if (residual && in) h[i] = add8(h[i], ld_v4(residual + base + 256 * i));
        }
        if (res_out) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (vec_of<V>(i, warp) < nv) *reinterpret_cast<uint4*>(res_out + base + 256 * i) = h[i];
        }
        float sum = sum_squares<V>(h);
        if (WARP_ROW) {
#pragma unroll
            for (int sh = 16; sh; sh >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, sh);
        } else {
            sum = cta_sum(sum, part, turn);
        }
        const float r = __frsqrt_rn(sum / (float)D + eps);
        if (rstd && vec_of<V>(0, warp) == 0) rstd[m] = r;
        norm_row<V, W>(h, g, r, base, nv, warp, y, q, s);
    }
}

// ---- gradient ------------------------------------------------------------------------------------
//
// With n = h r and g = gy w:  gx = r (g - n mean_d(g n)) + gres,  gw = sum_m gy n.
// The CTAs persist: each walks rows blockIdx.x, + gridDim.x, ..., keeps its share of gw in
// registers (fp32) and writes it to its row of the workspace; a second kernel adds the CTAs'
// rows in order: no atomics, the same bits every time.
//
// Bulk copies bring a CTA's next rows into a ring in shared memory while it works on one, so that
// the loads in flight do not depend on registers or on how the reductions serialise a row.  Stage
// s is refilled once the barrier inside the row's reduction has shown that every thread has read
// it.  A wait that runs out (see mxq_set_wait_limit_ns) ends the CTA: it stores no more rows, NaN
// as its share of gw, waits for its copies in flight, and is counted.
__device__ unsigned int g_norm_timeouts = 0;

constexpr uint64_t NORM_DRAIN_NS = 20000000000ull;
constexpr int NORM_MAX_STAGES = 4;

struct Ring {
    uint64_t full[NORM_MAX_STAGES];
    // whether a thread gave up its wait for the row, for rows in turn: a thread that is past the
    // row's barrier may give up the next one while others have yet to look at this one's
    int abort[2];
};

// N tensors' rows side by side in a stage of N * D bf16.
template <int N>
__device__ __forceinline__ void ring_fill(uint8_t* sm, Ring* ring, int st, const uint16_t* const (&from)[3], int64_t at,
                                          int D) {
    mbar_arrive_expect_tx(&ring->full[st], (uint32_t)(N * D * 2));
#pragma unroll
    for (int i = 0; i < N; ++i)
        bulk_load(sm + ((size_t)st * N + i) * D * 2, from[i] + at, (uint32_t)(D * 2), &ring->full[st]);
}

template <int N>
__device__ __forceinline__ void ring_start(uint8_t* sm, Ring* ring, int stages, const uint16_t* const (&from)[3],
                                           int64_t M, int D) {
    if (threadIdx.x == 0) {
        ring->abort[0] = ring->abort[1] = 0;
        for (int st = 0; st < stages; ++st) mbar_init(&ring->full[st], 1);
        for (int st = 0; st < stages; ++st) {
            const int64_t m = blockIdx.x + (int64_t)st * gridDim.x;
            if (m < M) ring_fill<N>(sm, ring, st, from, m * D, D);
        }
    }
    __syncthreads();
}

// After an abort at row m of stage st: thread 0 waits for the copies of the rows that were
// in flight (this one's and the stages' after it).
__device__ __forceinline__ void ring_leave(Ring* ring, int stages, int st, uint32_t phase, int64_t m, int64_t M) {
    if (threadIdx.x != 0) return;
    for (int i = 0; i < stages && m < M; ++i, m += gridDim.x) {
        mbar_wait_bounded(&ring->full[st], phase, NORM_DRAIN_NS);
        if (++st == stages) {
            st = 0;
            phase ^= 1;
        }
    }
    atomicAdd(&g_norm_timeouts, 1u);
}

// 16640 x 5120 with a residual's gradient: 104 us, 6.5 TB/s (the weights read again for every
// row: 127 us; without the ring: 227).
template <int V, typename W, bool RES>
__global__ void __launch_bounds__(512) rmsnorm_backward_kernel(
    const uint16_t* gy, const uint16_t* __restrict__ h, const W* __restrict__ w, const float* __restrict__ rstd,
    const uint16_t* gres, int64_t M, int D, uint16_t* gx, float* __restrict__ partial, uint64_t wait_ns, int stages) {
    constexpr int N = RES ? 3 : 2;
    extern __shared__ __align__(128) uint8_t norm_sm[];
    __shared__ Ring ring;
    __shared__ float part[64];
    grid_wait();
    const int tid = threadIdx.x, nv = D / 8;
    const uint16_t* const from[3] = {gy, h, gres};
    ring_start<N>(norm_sm, &ring, stages, from, M, D);
    W8<W> g[V] = {};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (vec_of<V>(i) < nv) g[i].load(w + 8 * vec_of<V>(i));
    f2 gw[V][4] = {};
    int st = 0, turn = 0;
    uint32_t phase = 0;
    const uint32_t row0 = smem_addr(norm_sm) + 16 * vec_of<V>(0);
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, turn ^= 1) {
        const int64_t base = m * D + 8 * vec_of<V>(0);
        const float r = __ldg(rstd + m);
        if (!mbar_wait_bounded(&ring.full[st], phase, wait_ns)) *(volatile int*)&ring.abort[turn] = 1;
        const uint32_t row = row0 + (uint32_t)(st * N * D * 2);
        uint4 a[V], b[V], e[V];
        f2 dot = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = vec_of<V>(i);
            a[i] = b[i] = e[i] = make_uint4(0, 0, 0, 0);
            if (v >= nv) continue;
            a[i] = lds_v4_at(row + 512 * i);
            b[i] = lds_v4_at(row + 2 * D + 512 * i);
            if (RES) e[i] = lds_v4_at(row + 4 * D + 512 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f2 f = bf2(word(a[i], j)), n = mul2(bf2(word(b[i], j)), f2{r, r});
                gw[i][j] = fma2(f, n, gw[i][j]);
                dot = fma2(mul2(f, g[i].pair(j)), n, dot);
            }
        }
        const float mean = cta_sum(dot.x + dot.y, part, turn, true) / (float)D;  // with a barrier: the stage is read
        if (*(volatile int*)&ring.abort[turn]) {
            // the weight's gradient lacks this CTA's rows: NaN in its share shows it
            const float nan = __int_as_float(0x7FC00000);
            for (int d = tid; d < D; d += (int)blockDim.x) partial[(int64_t)blockIdx.x * D + d] = nan;
            ring_leave(&ring, stages, st, phase, m, M);
            return;
        }
        if (tid == 0) {
            const int64_t next = m + (int64_t)stages * gridDim.x;
            if (next < M) ring_fill<N>(norm_sm, &ring, st, from, next * D, D);
        }
        if (++st == stages) {
            st = 0;
            phase ^= 1;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = vec_of<V>(i);
            if (v >= nv) continue;
            uint32_t o[4];
            const float k = -r * r * mean;  // r (f g - n mean) = f g r - h r^2 mean
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f2 t = mul2(mul2(bf2(word(a[i], j)), g[i].pair(j)), f2{r, r});
                t = fma2(bf2(word(b[i], j)), f2{k, k}, t);
                if (RES) t = fma2(bf2(word(e[i], j)), f2{1.0f, 1.0f}, t);
                o[j] = cvt_bf16x2(t.x, t.y);
            }
            *reinterpret_cast<uint4*>(gx + base + 256 * i) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    float* mine = partial + (int64_t)blockIdx.x * D;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = vec_of<V>(i);
        if (v >= nv) continue;
        *reinterpret_cast<float4*>(mine + 8 * v) = make_float4(gw[i][0].x, gw[i][0].y, gw[i][1].x, gw[i][1].y);
        *reinterpret_cast<float4*>(mine + 8 * v + 4) = make_float4(gw[i][2].x, gw[i][2].y, gw[i][3].x, gw[i][3].y);
    }
}

// gw[d] = sum over the n rows of partial, in a fixed order: warp i of the CTA adds rows
// i, i + 16, ..., then the sixteen sums are added in order.
constexpr int GW_WARPS = 16;
__global__ void __launch_bounds__(32 * GW_WARPS) rmsnorm_gw_kernel(const float* __restrict__ partial, int n, int D,
                                                                   float* __restrict__ gw) {
    __shared__ float sums[GW_WARPS][32];
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane;
    float v = 0.0f;
#pragma unroll 8
    for (int r = warp; r < n; r += GW_WARPS) v += partial[(int64_t)r * D + d];
    sums[warp][lane] = v;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int i = 1; i < GW_WARPS; ++i) v += sums[i][lane];
        gw[d] = v;
    }
}

constexpr int NORM_MAX_CTAS = 592;

// Four vectors per thread (fewer for short rows).
int norm_vectors(int nv) { return nv <= 32 ? 1 : nv <= 64 ? 2 : 4; }

// A ring kernel over M rows: two stages at first, as many CTAs per SM as then fit, and what
// shared memory they leave goes to more stages.  *grid: the CTAs launched (at most max_ctas).
template <typename K, typename... A>
cudaError_t launch_ring(K kernel, int v, int tensors, int64_t M, int D, int64_t max_ctas, unsigned* grid,
                        cudaStream_t stream, const A&... args) {
    const int nv = D / 8, threads = (nv + 32 * v - 1) / (32 * v) * 32;
    const int stage = tensors * D * 2;
    constexpr int TOTAL = 220 * 1024;  // of an SM, with the CTAs' own use (1.5 KB each) left aside
    constexpr int MAX_SMEM = TOTAL - 2048;
    static_assert(2 * 3 * 16384 * 2 <= MAX_SMEM, "two stages of the longest rows");
    // The attribute belongs to the kernel and not to the call, and other host threads launch it
    // and ask for its occupancy: always the same value, whatever this call takes.
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
    int per_sm = 0;
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, (size_t)2 * stage);
    if (e != cudaSuccess) return e;
    per_sm = std::max(1, per_sm);
    const int stages = std::max(2, std::min(NORM_MAX_STAGES, (TOTAL / per_sm - 2048) / stage));
    *grid = (unsigned)std::min({M, (int64_t)sm_count() * per_sm, max_ctas});
    return launch_dependent(kernel, *grid, threads, (size_t)stages * stage, stream, args..., stages);
}

template <typename W>
cudaError_t norm_forward(const uint16_t* x, const uint16_t* residual, const W* w, int64_t M, int D, float eps,
                         uint16_t* res_out, uint16_t* y, uint8_t* q, uint8_t* s, float* rstd, cudaStream_t stream) {
    const int nv = D / 8;
    const auto go = [&](auto kernel, int64_t grid, int threads) {
        return launch_dependent(kernel, (unsigned)std::min<int64_t>(grid, 0x7FFFFFFF), threads, 0, stream, x, residual,
                                w, M, D, eps, res_out, y, q, s, rstd);
    };
    const int64_t eighth = M / 8 + (M % 8 != 0);
    if (nv <= 32) return go(rmsnorm_mx_kernel<1, true, W>, eighth, 256);
    if (nv <= 64) return go(rmsnorm_mx_kernel<2, true, W>, eighth, 256);
    if (nv <= 128) return go(rmsnorm_mx_kernel<2, false, W>, M, (nv + 63) / 64 * 32);
    return go(rmsnorm_mx_kernel<4, false, W>, M, (nv + 127) / 128 * 32);
}

template <typename W>
cudaError_t norm_backward(const uint16_t* gy, const uint16_t* h, const W* w, const float* rstd, const uint16_t* gres,
                          int64_t M, int D, uint16_t* gx, float* gw, float* ws, cudaStream_t stream) {
    unsigned grid = 0;
    if (M > 0) {
        const int v = norm_vectors(D / 8);
        auto go = [&](auto vv) {
            constexpr int V = decltype(vv)::value;
            return gres ? launch_ring(rmsnorm_backward_kernel<V, W, true>, V, 3, M, D, NORM_MAX_CTAS, &grid, stream,
                                      gy, h, w, rstd, gres, M, D, gx, ws, wait_limit_ns())
                        : launch_ring(rmsnorm_backward_kernel<V, W, false>, V, 2, M, D, NORM_MAX_CTAS, &grid, stream,
                                      gy, h, w, rstd, gres, M, D, gx, ws, wait_limit_ns());
        };
        const cudaError_t e = v == 1   ? go(std::integral_constant<int, 1>())
                              : v == 2 ? go(std::integral_constant<int, 2>())
                                       : go(std::integral_constant<int, 4>());
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(rmsnorm_gw_kernel, (unsigned)(D / 32), 32 * GW_WARPS, 0, stream, ws, (int)grid, D, gw);
}

}  // namespace

unsigned int read_norm_timeouts() {
    unsigned int n = 0;
    if (cudaMemcpyFromSymbol(&n, g_norm_timeouts, sizeof(n)) != cudaSuccess) return 0xFFFFFFFFu;
    return n;
}

int64_t rmsnorm_workspace_bytes(int64_t M, int64_t D) { return 4 * D * std::min<int64_t>(M, NORM_MAX_CTAS); }

cudaError_t launch_rmsnorm_mx(const uint16_t* x, const uint16_t* residual, const void* w, bool w_bf16, int64_t M,
                              int D, float eps, uint16_t* res_out, uint16_t* y, uint8_t* q, uint8_t* s, float* rstd,
                              cudaStream_t stream) {
    return w_bf16 ? norm_forward(x, residual, static_cast<const uint16_t*>(w), M, D, eps, res_out, y, q, s, rstd,
                                 stream)
                  : norm_forward(x, residual, static_cast<const float*>(w), M, D, eps, res_out, y, q, s, rstd, stream);
}

cudaError_t launch_rmsnorm_backward(const uint16_t* gy, const uint16_t* h, const void* w, bool w_bf16,
                                    const float* rstd, const uint16_t* gres, int64_t M, int D, uint16_t* gx,
                                    float* gw, float* ws, cudaStream_t stream) {
    return w_bf16 ? norm_backward(gy, h, static_cast<const uint16_t*>(w), rstd, gres, M, D, gx, gw, ws, stream)
                  : norm_backward(gy, h, static_cast<const float*>(w), rstd, gres, M, D, gx, gw, ws, stream);
}

}  // namespace mxq
