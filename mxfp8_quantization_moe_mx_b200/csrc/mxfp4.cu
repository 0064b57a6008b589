// mxfp4.cu -- MXFP4 quantize and dequantize (sm_100a): 1x32 blocks of E2M1 codes, two to a
// byte (the even element in the low four bits), one E8M0 scale each.
//
//   b = clamp(floor(log2 amax) - 2, -127, 127) + 127  (the largest E2M1 value is 6 = 1.5 * 2^2),
//   code = satRNE_E2M1(x 2^(127 - b)); the product is exact in fp32 (a bf16 times a power
//   of two; where it is subnormal it lies under 2^-100 and rounds to 0 all the same).
//   A block holding Inf or NaN: b = 0xFF, codes 7 | sign (E2M1 has no NaN).
//
// Bound by HBM: 2 bytes in and 17/32 out per element.  One step per warp, four 16-byte
// vectors of bf16 per lane in it; a grid of persistent CTAs was slower in both directions, as
// were steps of one or two vectors.  (16, 8192, 5120): quantize 246 us (6.91 TB/s; persistent
// 273, two vectors 322), dequantize 252 us (6.73 TB/s; 301, 284).

#include <algorithm>

#include "dependent.cuh"
#include "mxq_launch.h"

namespace mxq {

namespace {

// E8M0 byte from the bf16 bits of the amax: E - 2 clamped at 0, 0xFF for Inf / NaN.
__device__ __forceinline__ uint32_t f4_scale_of_amax(uint32_t amax_bits) {
    const uint32_t E = amax_bits >> 7;
    return E == 255u ? 255u : (E > 2u ? E - 2u : 0u);
}

// Eight fp32 values -> eight E2M1 codes (a[0] in the lowest four bits), round to nearest
// even, saturating at 6.  cvt ... e2m1x2 puts its first source in the upper four bits.
__device__ __forceinline__ uint32_t cvt8_e2m1(const float (&a)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(a[0]), "f"(a[1]), "f"(a[2]), "f"(a[3]), "f"(a[4]), "f"(a[5]), "f"(a[6]), "f"(a[7]));
    return r;
}

// Eight bf16 values (one 16-byte vector) under scale byte b -> eight codes.
__device__ __forceinline__ uint32_t f4_codes8(const uint4& v, uint32_t b) {
    if (b == 255u) {
        // 7 | sign for each element
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t r = 0x77777777u;
#pragma unroll
        for (int i = 0; i < 4; ++i) r |= (((w[i] >> 15) & 1u) << (8 * i + 3)) | ((w[i] >> 31) << (8 * i + 7));
        return r;
    }
    const float m = mx_mult(b);
    float f[8];
    fmul2(bf16_lo(v.x), bf16_hi(v.x), m, m, f[0], f[1]);
    fmul2(bf16_lo(v.y), bf16_hi(v.y), m, m, f[2], f[3]);
    fmul2(bf16_lo(v.z), bf16_hi(v.z), m, m, f[4], f[5]);
    fmul2(bf16_lo(v.w), bf16_hi(v.w), m, m, f[6], f[7]);
    return cvt8_e2m1(f);
}

// The block maximum over the four lanes that hold a block.
__device__ __forceinline__ uint32_t block_amax(const uint4& v) {
    uint32_t m = mag2(amax2(amax2(v.x, v.y), amax2(v.z, v.w)));
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, __shfl_xor_sync(FULL_MASK, m, 1));
    return max(m, __shfl_xor_sync(FULL_MASK, m, 2));
}

// ---- flat blocks (plain scales): a warp's step = 8 U consecutive blocks, lane = part l % 4 of
// block u * 8 + l / 4
template <int U>
__global__ void __launch_bounds__(256) f4_quant_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ s, int64_t n_blocks) {
    grid_wait();
    const int lane = threadIdx.x & 31, part = lane & 3, sub = lane >> 2;
    const int64_t gwarp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t n_warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t base = gwarp * (8 * U); base < n_blocks; base += n_warps * (8 * U)) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t blk = base + u * 8 + sub;
            v[u] = blk < n_blocks ? ld_nc_v4(x + blk * 32 + part * 8) : make_uint4(0, 0, 0, 0);
        }
        uint32_t mine = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t blk = base + u * 8 + sub;
            const uint32_t b = f4_scale_of_amax(block_amax(v[u]));
            const uint32_t c = f4_codes8(v[u], b);
            if (blk < n_blocks) *reinterpret_cast<uint32_t*>(q + blk * 16 + part * 4) = c;
            const uint32_t t = __shfl_sync(FULL_MASK, b, (lane & 7) * 4);
            if ((lane >> 3) == u) mine = t;
        }
        if (lane < 8 * U && base + lane < n_blocks) s[base + lane] = (uint8_t)mine;
    }
}

// ---- with scales in the tensor cores' tiles: a CTA per padded 128-row tile x 512 columns
// (16 scale columns, 4 scale tiles).  Warp w takes rows w, w + 8, ... of the tile, 1024
// bytes of a row per step; scales gather in shared memory and leave as whole 16-byte lines.
// 16411 x 5120 over 16 groups: 45 us, 4.7 TB/s (plain scales 33).  What it lacks to a copy is each
// CTA's search for its group, before its first load: CTAs of a quarter of this took 59 us, four
// rows a step (fewer CTAs at a time) 54, one row 50.  Five CTAs per SM leave 48 registers, of
// which 32 bytes a thread are spilled.
__global__ void __launch_bounds__(256, 5) f4_quant_blocked_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                               int64_t cols, uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ s, uint8_t* __restrict__ sf,
                                                               const int32_t* __restrict__ offs, int32_t G,
                                                               int64_t tiles_per_matrix, int chunks) {
    __shared__ __align__(16) uint8_t sc[128][16];
    __shared__ int64_t info[2];  // first source row of the tile, valid rows in it (-1: no tile)
    grid_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t tile = blockIdx.x / (unsigned)chunks;  // a tile's chunks side by side
    const int chunk = (int)(blockIdx.x % (unsigned)chunks);
    if (G <= 0) {
        if (tid == 0) {
            const int64_t b = tile / tiles_per_matrix, i = tile % tiles_per_matrix;
            info[0] = b * rows + i * 128;
            info[1] = min((int64_t)128, rows - i * 128);
        }
    } else if (warp == 0) {
        if (lane == 0) info[1] = -1;
        __syncwarp();
        int run = 0;
        int64_t padded = 0;
        bool found = false;
        for (int h0 = 0; h0 < G && !found; h0 += 32) {
            const int h = h0 + lane;
            int e = h < G ? max(offs[h], 0) : 0;
#pragma unroll
            for (int sh = 1; sh < 32; sh <<= 1) {
                const int o = __shfl_up_sync(FULL_MASK, e, sh);
                if (lane >= sh) e = max(e, o);
            }
            e = max(e, run);
            const int up = __shfl_up_sync(FULL_MASK, e, 1);
            const int prev_e = lane == 0 ? run : up;
            const int64_t end = min((int64_t)e, rows), start = min((int64_t)prev_e, rows);
            const int64_t n_tiles = h < G ? (end - start + 127) / 128 : 0;
            int64_t inc = n_tiles;
#pragma unroll
            for (int sh = 1; sh < 32; sh <<= 1) {
                const int64_t o = __shfl_up_sync(FULL_MASK, inc, sh);
                if (lane >= sh) inc += o;
            }
            const int64_t first = padded + inc - n_tiles;
            const bool mine = h < G && tile >= first && tile < first + n_tiles;
            if (mine) {
                info[0] = start + (tile - first) * 128;
                info[1] = min((int64_t)128, end - info[0]);
            }
            found = __any_sync(FULL_MASK, mine);
            padded += __shfl_sync(FULL_MASK, inc, 31);
            run = __shfl_sync(FULL_MASK, e, 31);
        }
    }
    for (int i = tid; i < 128; i += 256) *reinterpret_cast<uint4*>(sc[i]) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const int64_t r0 = info[0], valid = info[1];
    if (valid < 0) return;
    const int64_t c0 = (int64_t)chunk * 512;
    const int64_t n_k = cols / 32;
    constexpr int R = 2;  // rows of a warp in flight
    for (int rr = warp; rr < valid; rr += 8 * R) {
        uint4 v[R][2];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t c = c0 + u * 256 + lane * 8;
                const int r = rr + 8 * i;
                v[i][u] = r < valid && c < cols ? ld_nc_v4(x + (r0 + r) * cols + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t c = c0 + u * 256 + lane * 8;
                const int r = rr + 8 * i;
                const uint32_t b = f4_scale_of_amax(block_amax(v[i][u]));
                const uint32_t code = f4_codes8(v[i][u], b);
                if (r < valid && c < cols) {
                    *reinterpret_cast<uint32_t*>(q + ((r0 + r) * cols + c) / 2) = code;
                    if ((lane & 3) == 0) {
                        sc[r][u * 8 + (lane >> 2)] = (uint8_t)b;
                        if (s) s[(r0 + r) * n_k + c / 32] = (uint8_t)b;
                    }
                }
            }
    }
    __syncthreads();
    if (tid < 128) {
        const int64_t col_tiles = (n_k + 3) / 4;
        const int j = tid >> 5;  // scale tile of this CTA's four
        const int64_t ct = (int64_t)chunk * 4 + j;
        if (ct < col_tiles) {
            uint32_t w[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) w[a] = *reinterpret_cast<const uint32_t*>(&sc[32 * a + lane][4 * j]);
            *reinterpret_cast<uint4*>(sf + (tile * col_tiles + ct) * 512 + lane * 16) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---- dequantize: a lane per 8 elements (4 bytes of codes -> one 16-byte store), U steps of
// a warp in flight

// Two codes (the low byte) as fp32, through a packed pair of f16, exactly.
__device__ __forceinline__ void e2m1x2_to_f32(uint32_t byte, float& a, float& b) {
    asm("{\n\t.reg .b8 c;\n\t.reg .b32 p, t;\n\t.reg .b16 h0, h1;\n\t"
        "mov.b32 {c, _, _, _}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 p, c;\n\t"
        "mov.b32 {h0, h1}, p;\n\t"
        "cvt.f32.f16 %0, h0;\n\t"
        "cvt.f32.f16 %1, h1;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(byte));
}

__device__ __forceinline__ uint4 f4_dequant8(uint32_t codes, uint32_t b) {
    if (b == 255u) return make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
    const float sc = e8m0_value(b);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f0, f1, p0, p1;
        e2m1x2_to_f32((codes >> (8 * i)) & 0xFFu, f0, f1);
        fmul2(f0, f1, sc, sc, p0, p1);
        o[i] = cvt_bf16x2(p0, p1);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int U>
__global__ void __launch_bounds__(256) f4_dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                         uint16_t* __restrict__ y, int64_t n8) {
    grid_wait();
    const int lane = threadIdx.x & 31;
    const int64_t gwarp = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), n_warps = (int64_t)gridDim.x * 8;
    for (int64_t base = gwarp * (32 * U); base < n8; base += n_warps * (32 * U)) {
        uint32_t c[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = base + 32 * u + lane;
            c[u] = i < n8 ? __ldg(reinterpret_cast<const uint32_t*>(q) + i) : 0u;
            b[u] = i < n8 ? ld_nc_u8(s + (i >> 2)) : 0u;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = base + 32 * u + lane;
            if (i < n8) reinterpret_cast<uint4*>(y)[i] = f4_dequant8(c[u], b[u]);
        }
    }
}

}  // namespace

cudaError_t launch_f4_quant(const uint16_t* x, int64_t batch, int64_t rows, int64_t cols, uint8_t* q, uint8_t* s,
                            uint8_t* sf, const int32_t* offs, int32_t G, cudaStream_t stream) {
    if (!sf) {
        constexpr int U = 4;
        const int64_t n_blocks = batch * rows * (cols / 32);
        const int64_t ctas = (n_blocks + 8 * 8 * U - 1) / (8 * 8 * U);
        return launch_dependent(f4_quant_kernel<U>, (unsigned)std::min<int64_t>(ctas, 0x7FFFFFFF), 256, 0, stream, x,
                                q, s, n_blocks);
    }
    const int64_t per = (rows + 127) / 128;
    const int64_t tiles = G > 0 ? (rows + 127 * (int64_t)G) / 128 : batch * per;
    const int64_t chunks = (cols + 511) / 512;
    if (tiles <= 0 || chunks <= 0) return cudaSuccess;
    if (tiles > 0x7FFFFFFFLL / chunks) return cudaErrorInvalidConfiguration;
    return launch_dependent(f4_quant_blocked_kernel, (unsigned)(tiles * chunks), 256, 0, stream, x, rows, cols, q, s,
                            sf, offs, G, per, (int)chunks);
}

cudaError_t launch_f4_dequant(const uint8_t* q, const uint8_t* s, uint16_t* y, int64_t n, cudaStream_t stream) {
    constexpr int U = 4;
    const int64_t n8 = n / 8;
    const int64_t ctas = (n8 + 256 * U - 1) / (256 * U);
    return launch_dependent(f4_dequant_kernel<U>, (unsigned)std::min<int64_t>(ctas, 0x7FFFFFFF), 256, 0, stream, q, s,
                            y, n8);
}

}  // namespace mxq
