// rmsnorm.cu -- residual addition, root-mean-square norm and MXFP8 quantization in one
// pass, and the norm's gradient (sm_100a).
//
//   h = bf16(x + residual)            (x itself without a residual)
//   r = 1 / sqrt(mean_d h^2 + eps)    (fp32)
//   y = bf16(h r w)
//   q, s = 1x32 MXFP8 blocks of y     (the bytes mx_quantize gives for y)
//
// Everything is bound by HBM: a row is read once, stays in registers through the two
// reductions (sum of squares over the CTA, block maxima over four lanes) and leaves as
// codes.  A CTA owns a row at a time; thread t holds the 8-element vectors t, t + T, ...,
// so four neighbouring lanes hold one 32-element block.  The sums are fp32: a thread adds
// at most 32 squares, then 5 shuffle steps and at most 32 warps' sums, so the relative
// error stays under 2^-18.

#include <algorithm>
#include <type_traits>

#include "mxq_device.cuh"
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

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                      cvt_bf16x2(f[6], f[7]));
}

// Eight consecutive weights as fp32.
__device__ __forceinline__ void load_w8(const float* w, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w)), b = __ldg(reinterpret_cast<const float4*>(w) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load_w8(const uint16_t* w, float (&f)[8]) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(w)), f);
}

// Sum over the CTA, returned to every thread.  `part` holds 2 x 32 floats; `turn`
// alternates between calls, so that one barrier a call is enough.
__device__ __forceinline__ float cta_sum(float v, float* part, int turn) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(FULL_MASK, v, s);
    if (n == 1) return v;
    if (lane == 0) part[32 * turn + warp] = v;
    __syncthreads();
    v = lane < n ? part[32 * turn + lane] : 0.0f;
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(FULL_MASK, v, s);
    return v;
}

// V 8-element vectors per thread; D / 8 <= V * blockDim.x.
template <int V, typename W>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512) rmsnorm_mx_kernel(
    const uint16_t* x, const uint16_t* residual, const W* __restrict__ w, int64_t M, int D, float eps,
    uint16_t* res_out, uint16_t* y, uint8_t* __restrict__ q, uint8_t* __restrict__ s, float* __restrict__ rstd) {
    __shared__ float part[64];
    const int tid = threadIdx.x, T = blockDim.x, nv = D / 8;
    int turn = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, turn ^= 1) {
        const int64_t at = m * D;
        uint4 h[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * T;
            h[i] = v < nv ? ld_v4(x + at + 8 * v) : make_uint4(0, 0, 0, 0);
        }
        if (residual) {
            uint4 a[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = tid + i * T;
                a[i] = v < nv ? ld_v4(residual + at + 8 * v) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[8], g[8];
                unpack8(h[i], f);
                unpack8(a[i], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += g[j];
                h[i] = pack8(f);
            }
        }
        if (res_out) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = tid + i * T;
                if (v < nv) *reinterpret_cast<uint4*>(res_out + at + 8 * v) = h[i];
            }
        }
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[8];
            unpack8(h[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fmaf(f[j], f[j], sq);
        }
        const float r = __frsqrt_rn(cta_sum(sq, part, turn) / (float)D + eps);
        if (rstd && tid == 0) rstd[m] = r;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * T;
            float f[8], g[8];
            unpack8(h[i], f);
            if (v < nv) load_w8(w + 8 * v, g);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * r * g[j];
            const uint4 o = pack8(f);
            uint32_t am = mag2(amax2(amax2(o.x, o.y), amax2(o.z, o.w)));
            am = max(am & 0xFFFFu, am >> 16);
            am = max(am, __shfl_xor_sync(FULL_MASK, am, 1));
            am = max(am, __shfl_xor_sync(FULL_MASK, am, 2));
            const uint32_t b = e8m0_of_amax(am);
            uint2 c;
            if (b != 255u) {
                const float mul = mx_mult(b);
                c.x = quant4(o.x, o.y, mul);
                c.y = quant4(o.z, o.w, mul);
            } else {
                c.x = nan4(o.x, o.y);
                c.y = nan4(o.z, o.w);
            }
            if (v < nv) {
                if (y) *reinterpret_cast<uint4*>(y + at + 8 * v) = o;
                *reinterpret_cast<uint2*>(q + at + 8 * v) = c;
                if ((v & 3) == 0) s[(at >> 5) + (v >> 2)] = (uint8_t)b;
            }
        }
    }
}

// ---- gradient ------------------------------------------------------------------------------------
//
// With n = h r and g = gy w:  gx = r (g - n mean_d(g n)) + gres,  gw = sum_m gy n.
// A CTA walks rows blockIdx.x, + gridDim.x, ... and keeps its share of gw in registers
// (fp32), writes it to its row of the workspace, and a second kernel adds the CTAs' rows in
// order: no atomics, the same bits every time.
template <int V, typename W>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512) rmsnorm_backward_kernel(
    const uint16_t* gy, const uint16_t* __restrict__ h, const W* __restrict__ w, const float* __restrict__ rstd,
    const uint16_t* gres, int64_t M, int D, uint16_t* gx, float* __restrict__ partial) {
    __shared__ float part[64];
    const int tid = threadIdx.x, T = blockDim.x, nv = D / 8;
    float gw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) gw[i][j] = 0.0f;
    int turn = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, turn ^= 1) {
        const int64_t at = m * D;
        uint4 a[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * T;
            a[i] = v < nv ? ld_v4(gy + at + 8 * v) : make_uint4(0, 0, 0, 0);
            b[i] = v < nv ? ld_nc_v4(h + at + 8 * v) : make_uint4(0, 0, 0, 0);
        }
        const float r = __ldg(rstd + m);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * T;
            float f[8], n[8], g[8];
            unpack8(a[i], f);
            unpack8(b[i], n);
            if (v < nv) load_w8(w + 8 * v, g);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[j] *= r;
                gw[i][j] = fmaf(f[j], n[j], gw[i][j]);
                dot = fmaf(f[j] * g[j], n[j], dot);
            }
        }
        const float mean = cta_sum(dot, part, turn) / (float)D;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * T;
            if (v >= nv) continue;
            float f[8], n[8], g[8], o[8];
            unpack8(a[i], f);
            unpack8(b[i], n);
            load_w8(w + 8 * v, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = r * (f[j] * g[j] - n[j] * r * mean);
            if (gres) {
                unpack8(ld_v4(gres + at + 8 * v), f);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += f[j];
            }
            *reinterpret_cast<uint4*>(gx + at + 8 * v) = pack8(o);
        }
    }
    float* mine = partial + (int64_t)blockIdx.x * D;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = tid + i * T;
        if (v >= nv) continue;
        *reinterpret_cast<float4*>(mine + 8 * v) = make_float4(gw[i][0], gw[i][1], gw[i][2], gw[i][3]);
        *reinterpret_cast<float4*>(mine + 8 * v + 4) = make_float4(gw[i][4], gw[i][5], gw[i][6], gw[i][7]);
    }
}

// gw[d] = sum over the n rows of partial, in a fixed order: warp y of the CTA adds rows
// y, y + 8, ..., then the eight sums are added in order.
__global__ void __launch_bounds__(256) rmsnorm_gw_kernel(const float* __restrict__ partial, int n, int D,
                                                         float* __restrict__ gw) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane;
    float v = 0.0f;
    for (int r = warp; r < n; r += 8) v += partial[(int64_t)r * D + d];
    sums[warp][lane] = v;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += sums[i][lane];
        gw[d] = v;
    }
}

struct NormShape {
    int v, threads;
};

// Threads and vectors per thread for a row of D elements: one vector per thread while that
// fits in 1024 threads and rows are few, more per thread otherwise.
NormShape norm_shape(int64_t M, int D) {
    const int nv = D / 8;
    const int v = nv <= 32 ? 1 : nv <= 1024 && M <= 2 * (int64_t)sm_count() ? 1 : nv <= 64 ? 2 : 4;
    const int per = (nv + v - 1) / v;
    return {v, (per + 31) / 32 * 32};  // at most 1024 for v = 1, 512 for v = 4 (D <= 16384)
}

constexpr int NORM_MAX_CTAS = 592;

}  // namespace

int64_t rmsnorm_workspace_bytes(int64_t M, int64_t D) { return 4 * D * std::min<int64_t>(M, NORM_MAX_CTAS); }

cudaError_t launch_rmsnorm_mx(const uint16_t* x, const uint16_t* residual, const void* w, bool w_bf16, int64_t M,
                              int D, float eps, uint16_t* res_out, uint16_t* y, uint8_t* q, uint8_t* s, float* rstd,
                              cudaStream_t stream) {
    const NormShape sh = norm_shape(M, D);
    const int per_sm = std::max(1, 1536 / sh.threads);
    const unsigned grid = (unsigned)std::min<int64_t>(M, (int64_t)sm_count() * per_sm);
    auto go = [&](auto vv) {
        constexpr int V = decltype(vv)::value;
        if (w_bf16)
            rmsnorm_mx_kernel<V, uint16_t><<<grid, sh.threads, 0, stream>>>(
                x, residual, static_cast<const uint16_t*>(w), M, D, eps, res_out, y, q, s, rstd);
        else
            rmsnorm_mx_kernel<V, float><<<grid, sh.threads, 0, stream>>>(x, residual, static_cast<const float*>(w), M,
                                                                         D, eps, res_out, y, q, s, rstd);
        return cudaGetLastError();
    };
    switch (sh.v) {
        case 1: return go(std::integral_constant<int, 1>());
        case 2: return go(std::integral_constant<int, 2>());
        default: return go(std::integral_constant<int, 4>());
    }
}

cudaError_t launch_rmsnorm_backward(const uint16_t* gy, const uint16_t* h, const void* w, bool w_bf16,
                                    const float* rstd, const uint16_t* gres, int64_t M, int D, uint16_t* gx,
                                    float* gw, float* ws, cudaStream_t stream) {
    if (M > 0) {
        const NormShape sh = norm_shape(M, D);
        const int per_sm = std::max(1, std::min(4, 1024 / sh.threads));
        const unsigned grid = (unsigned)std::min({M, (int64_t)sm_count() * per_sm, (int64_t)NORM_MAX_CTAS});
        auto go = [&](auto vv) {
            constexpr int V = decltype(vv)::value;
            if (w_bf16)
                rmsnorm_backward_kernel<V, uint16_t><<<grid, sh.threads, 0, stream>>>(
                    gy, h, static_cast<const uint16_t*>(w), rstd, gres, M, D, gx, ws);
            else
                rmsnorm_backward_kernel<V, float><<<grid, sh.threads, 0, stream>>>(
                    gy, h, static_cast<const float*>(w), rstd, gres, M, D, gx, ws);
            return cudaGetLastError();
        };
        cudaError_t e;
        switch (sh.v) {
            case 1: e = go(std::integral_constant<int, 1>()); break;
            case 2: e = go(std::integral_constant<int, 2>()); break;
            default: e = go(std::integral_constant<int, 4>()); break;
        }
        if (e != cudaSuccess) return e;
        rmsnorm_gw_kernel<<<(unsigned)(D / 32), 256, 0, stream>>>(ws, (int)grid, D, gw);
    } else {
        rmsnorm_gw_kernel<<<(unsigned)(D / 32), 256, 0, stream>>>(ws, 0, D, gw);
    }
    return cudaGetLastError();
}

}  // namespace mxq
