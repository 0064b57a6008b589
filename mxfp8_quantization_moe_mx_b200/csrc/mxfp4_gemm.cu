// mxfp4_gemm.cu -- MXFP4 grouped GEMM on the 5th-generation tensor cores (sm_100a).
//
// For the rows m of expert group g (the offsets' clamp rule),
//     out[m][n] = sum_k  A[m][k] 2^(sa[m][k/32]-127)  *  B[g][n][k] 2^(sb[g][n][k/32]-127)
// with A (M, K) and B (G, N, K) E2M1 codes, two to a byte, and E8M0 scales of 1x32 blocks in
// the 128 x 4 tiles of mx_scales_to_blocked.  tcgen05.mma.kind::mxf4.block_scale with K = 64
// and two scales per row and MMA (scale_vec::2X), fp32 accumulation in tensor memory, bf16
// output.  A stage of the ring is 256 elements = 128 bytes of every operand row and two
// scale tiles of 128 rows; K % 256 == 128 ends with half a stage: its second half is zero
// fill, and its MMAs are not issued (zero codes under a neighbour's NaN scale would be NaN).
//
// Two kernels, chosen by the rows a group has on average (see use_narrow):
//   wide    a 256 x 256 unit per CTA pair (tcgen05 .cta_group::2): the tokens are the MMA's
//           M side.  Bound by the tensor cores; a group's last unit costs as much as a full
//           one.
//   narrow  a unit is 128 weight rows x up to 128 tokens on one CTA: the weights are the M
//           side, so few tokens cost few MMA columns (N = 32, 64, 96 or 128, set per unit in
//           the instruction descriptor) and the kernel streams the weights at the rate of
//           HBM.  Only the 8- or 32-row pieces of the token tile that hold rows of the group
//           are loaded.  A unit's tokens always begin a 128-row scale tile: the MMA takes a
//           scale address only at the first of a tile's four tensor-memory columns.
// Both are persistent, with one producer lane (TMA), one MMA lane, four epilogue warps, and
// every wait bounded as in the MXFP8 kernel (mxq_wait_timeouts counts CTAs that gave up).

#include <algorithm>
#include <cstring>

#include "mxq_launch.h"
#include "tc_pair.cuh"

namespace mxq {

__device__ unsigned int g_f4_gemm_timeouts = 0;  // CTAs that gave up a bounded wait

namespace {

constexpr int F4_BKB = 128;                  // bytes of an operand row per stage
constexpr int F4_BK = 256;                   // elements
constexpr int F4_ROWS = 128;
constexpr int F4_TILE = F4_ROWS * F4_BKB;    // 16 KB
constexpr int F4_SF = 1024;                  // two 128 x 4 scale tiles

// ---- wide: 256 x 256 per CTA pair --------------------------------------------------------------

constexpr int FW_BN = 256;
constexpr int FW_STAGES = 6;
constexpr int FW_OFF_B = FW_STAGES * F4_TILE;
constexpr int FW_OFF_SFA = FW_OFF_B + FW_STAGES * F4_TILE;
constexpr int FW_OFF_SFB = FW_OFF_SFA + FW_STAGES * F4_SF;
constexpr int FW_SMEM = FW_OFF_SFB + FW_STAGES * 2 * F4_SF + 1024;  // + alignment slack
constexpr uint32_t FW_CTA_TX = 2 * F4_TILE + 3 * F4_SF;             // one CTA's bytes per stage
constexpr uint32_t FW_TMEM_SFA = 256;                               // 8 columns per stage
constexpr uint32_t FW_TMEM_SFB = 256 + 8 * FW_STAGES;               // 16 columns per stage
static_assert(FW_TMEM_SFB + 16 * FW_STAGES <= 512, "tensor-memory columns");
static_assert(FW_SMEM <= 227 * 1024, "shared memory per CTA");

__device__ __forceinline__ void mma_f4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}

// Instruction descriptor of kind::mxf4: E2M1 A and B, E8M0 scales, an M x N tile; `id` the
// first of the two scale bytes (0 or 2) of the A and B scale columns.
template <int M>
__device__ __forceinline__ uint32_t idesc_f4(uint32_t n, uint32_t id) {
    constexpr uint32_t base = 1u << 7 | 1u << 10 | 1u << 23 | (uint32_t)(M >> 4) << 24;
    return base | (n >> 3) << 17 | id << 4 | id << 29;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(192, 1) f4_gemm_wide_kernel(
    const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
    const __grid_constant__ CUtensorMap sfamap, const __grid_constant__ CUtensorMap sfbmap,
    const int32_t* __restrict__ offs, int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* __restrict__ out) {
    extern __shared__ uint8_t dyn_smem[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[FW_STAGES], empty[FW_STAGES], acc_full, acc_empty, drained;
    __shared__ uint32_t tmem_base_s;
    __shared__ uint32_t issued_s[2];  // stages each CTA's producer armed / issued (exchanged at the end)
    __shared__ int64_t n_work_s;
    __shared__ int abort_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const bool first = rank == 0;
    const int64_t cl = blockIdx.x >> 1, n_cl = gridDim.x >> 1;
    const int64_t n_tiles_n = N / FW_BN;
    const int64_t k_blocks = (K + F4_BK - 1) / F4_BK;
    const int64_t col_tiles = K / 128;

    if (warp == 0) {
        PairTile pt;
        int64_t total;
        gg_find_pair(offs, G, M, -1, &pt, &total);
        if (lane == 0) {
            n_work_s = total * n_tiles_n;
            abort_s = 0;
            issued_s[0] = issued_s[1] = 0;
            for (int s = 0; s < FW_STAGES; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            mbar_init(&acc_full, 1);
            mbar_init(&acc_empty, 8);  // the epilogue warps of both CTAs
            mbar_init(&drained, 1);
        }
    }
    if (warp == 1) tmem_alloc_pair(&tmem_base_s, 512);
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers are initialised before either signals the other's
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int64_t n_work = n_work_s;
    const uint32_t full0 = cluster_map(&full[0], 0);  // the first CTA's `full` ring (8 bytes apart)
    const uint32_t acc_empty0 = cluster_map(&acc_empty, 0);

    uint32_t it_prod = 0;
    if (warp == 0) {
        // ---- producer (both CTAs)
        const uint64_t pol = l2_policy_evict_last();
        bool stop = false;
        for (int64_t w = cl; w < n_work && !stop; w += n_cl) {
            const int64_t p = w / n_tiles_n, n0 = (w % n_tiles_n) * FW_BN;
            PairTile pt;
            gg_find_pair(offs, G, M, p, &pt, nullptr);
            if (lane == 0) {
                const int64_t my_row = pt.row0 + (int64_t)rank * F4_ROWS;
                const int64_t my_mt = (rank == 1 && pt.valid1 > 0) ? pt.mt0 + 1 : pt.mt0;  // filler: any real tile
                const int64_t sfa_row = 2 * my_mt * col_tiles;
                const int64_t sfb_row = 2 * ((int64_t)pt.g * (N / 128) + n0 / 128) * col_tiles;
                const int b_row = (int)((int64_t)pt.g * N + n0 + (int64_t)rank * (FW_BN / 2));
                for (int64_t kb = 0; kb < k_blocks; ++kb, ++it_prod) {
                    const int s = (int)(it_prod % FW_STAGES);
                    const uint32_t r = it_prod / FW_STAGES;
                    if (!mbar_wait_bounded(&empty[s], (r & 1) ^ 1, GG_WAIT_NS) || *(volatile int*)&abort_s) {
                        atomicExch(&abort_s, 1);
                        stop = true;
                        break;
                    }
                    if (first) mbar_arrive_expect_tx(&full[s], 2 * FW_CTA_TX);
                    const uint32_t bar = full0 + 8u * (uint32_t)s;
                    tma_load_2d_pair(sm + s * F4_TILE, &amap, (int)(kb * F4_BKB), (int)my_row, bar, pol);
                    tma_load_2d_pair(sm + FW_OFF_B + s * F4_TILE, &bmap, (int)(kb * F4_BKB), b_row, bar, pol);
                    tma_load_2d_pair(sm + FW_OFF_SFA + s * F4_SF, &sfamap, 0, (int)(sfa_row + 4 * kb), bar, pol);
                    tma_load_2d_pair(sm + FW_OFF_SFB + s * 2 * F4_SF, &sfbmap, 0, (int)(sfb_row + 4 * kb), bar, pol);
                    tma_load_2d_pair(sm + FW_OFF_SFB + s * 2 * F4_SF + F4_SF, &sfbmap, 0,
                                     (int)(sfb_row + 2 * col_tiles + 4 * kb), bar, pol);
                }
            }
            stop = __shfl_sync(FULL_MASK, stop ? 1 : 0, 0) != 0;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer (the first CTA)
        if (first && lane == 0) {
            uint32_t it = 0;
            int64_t i = 0;
            for (int64_t w = cl; w < n_work; w += n_cl, ++i) {
                if (i > 0 && !mbar_wait_bounded(&acc_empty, (uint32_t)((i - 1) & 1), GG_WAIT_NS)) {
                    atomicExch(&abort_s, 1);
                    break;
                }
                tc_fence_after();
                bool ok = true;
                for (int64_t kb = 0; kb < k_blocks; ++kb, ++it) {
                    const int s = (int)(it % FW_STAGES);
                    const uint32_t r = it / FW_STAGES;
                    if (!mbar_wait_bounded(&full[s], r & 1, GG_WAIT_NS) || *(volatile int*)&abort_s) {
                        atomicExch(&abort_s, 1);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // scale columns: A [scale tile][4], B [scale tile][column half][4]
                    const uint32_t t_sfa = tmem + FW_TMEM_SFA + 8 * s, t_sfb = tmem + FW_TMEM_SFB + 16 * s;
                    const uint8_t* sfa = sm + FW_OFF_SFA + s * F4_SF;
                    const uint8_t* sfb = sm + FW_OFF_SFB + s * 2 * F4_SF;
                    tmem_cp_sf_pair(t_sfa, desc_sf(sfa));
                    tmem_cp_sf_pair(t_sfb, desc_sf(sfb));
                    tmem_cp_sf_pair(t_sfb + 4, desc_sf(sfb + F4_SF));
                    tmem_cp_sf_pair(t_sfa + 4, desc_sf(sfa + 512));
                    tmem_cp_sf_pair(t_sfb + 8, desc_sf(sfb + 512));
                    tmem_cp_sf_pair(t_sfb + 12, desc_sf(sfb + F4_SF + 512));
                    const uint64_t a0 = desc_sw128(sm + s * F4_TILE), b0 = desc_sw128(sm + FW_OFF_B + s * F4_TILE);
                    const uint32_t nk = K - kb * F4_BK >= F4_BK ? 4 : 2;
                    for (uint32_t k = 0; k < nk; ++k) {  // K = 64 per MMA: 32 bytes further along the swizzled rows
                        const uint32_t id = 2 * (k & 1), t = k >> 1;
                        mma_f4_pair(tmem, a0 + 2 * k, b0 + 2 * k, idesc_f4<256>(FW_BN, id),
                                    (t_sfa + 4 * t) | id << 30, (t_sfb + 8 * t) | id << 30,
                                    (kb > 0 || k > 0) ? 1u : 0u);
                    }
                    mma_commit_both(&empty[s]);  // the stage is free in both CTAs once these MMAs have read it
                }
                if (!ok) break;              // a partial accumulator is never handed to the epilogues
                mma_commit_both(&acc_full);  // the unit's accumulators are complete once its MMAs are
            }
            // every tcgen05 operation issued above (and its arrivals) is done before the pair
            // frees tensor memory or leaves
            mma_commit_own(&drained);
            if (!mbar_wait_bounded(&drained, 0, GG_DRAIN_NS)) atomicExch(&abort_s, 1);
        }
        __syncwarp();
    } else {
        // ---- epilogue (both CTAs): warp w reads accumulator lanes (rows) 32 (w % 4) .. + 31
        const int quarter = warp & 3;
        const int r = 32 * quarter + lane;
        int64_t i = 0;
        for (int64_t w = cl; w < n_work; w += n_cl, ++i) {
            const int64_t p = w / n_tiles_n, n0 = (w % n_tiles_n) * FW_BN;
            PairTile pt;
            gg_find_pair(offs, G, M, p, &pt, nullptr);
            const bool done = mbar_wait_bounded(&acc_full, (uint32_t)(i & 1), GG_WAIT_NS);
            if (!done) atomicExch(&abort_s, 1);
            if (__any_sync(FULL_MASK, !done) || *(volatile int*)&abort_s) break;
            tc_fence_after();
            // the whole row, rounded to bf16 in registers, so the accumulator is released
            // before the stores and the next unit's MMAs overlap them
            uint32_t v16[FW_BN / 2];
#pragma unroll
            for (int c0 = 0; c0 < FW_BN; c0 += 32) {
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)c0, v);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v16[c0 / 2 + j] = cvt_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty0);  // this warp's quarter is read
            const int64_t valid = rank == 0 ? pt.valid0 : pt.valid1;
            if (r < valid) {
                uint4* orow = reinterpret_cast<uint4*>(out + (pt.row0 + (int64_t)rank * F4_ROWS + r) * N + n0);
#pragma unroll
                for (int q = 0; q < FW_BN / 8; ++q)
                    orow[q] = make_uint4(v16[4 * q], v16[4 * q + 1], v16[4 * q + 2], v16[4 * q + 3]);
            }
        }
    }

    // ---- leaving: account every copy either producer started on the first CTA's `full`
    // barriers and wait for them there, so neither CTA's shared memory is still a copy's
    // destination (or a barrier still to be signalled) when the pair exits
    if (warp == 0 && lane == 0) {
        issued_s[rank] = it_prod;
        st_cluster_u32(cluster_map(&issued_s[rank], rank ^ 1u), it_prod);
    }
    tc_fence_before();
    cluster_sync();
    if (first && warp == 0 && lane == 0) {
        const uint32_t i0 = issued_s[0], i1 = issued_s[1];
        // stages the second CTA filled but this one never armed: arm them for its bytes;
        // stages armed for both but filled only here: count the missing bytes as arrived
        for (uint32_t i = i0; i < i1; ++i) mbar_arrive_expect_tx(&full[i % FW_STAGES], FW_CTA_TX);
        for (uint32_t i = i1; i < i0; ++i) mbar_complete_tx(&full[i % FW_STAGES], FW_CTA_TX);
        const uint32_t hi = max(i0, i1);
        for (uint32_t i = hi > (uint32_t)FW_STAGES ? hi - FW_STAGES : 0u; i < hi; ++i)
            if (!mbar_wait_bounded(&full[i % FW_STAGES], (i / FW_STAGES) & 1, GG_DRAIN_NS)) atomicExch(&abort_s, 1);
    }
    tc_fence_before();
    __syncthreads();
    if (abort_s && tid == 0) atomicAdd(&g_f4_gemm_timeouts, 1u);
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ---- narrow: 128 weight rows x up to 128 tokens per CTA ----------------------------------------

constexpr int FN_STAGES = 6;
constexpr int FN_OFF_T = FN_STAGES * F4_TILE;
constexpr int FN_OFF_SFW = FN_OFF_T + FN_STAGES * F4_TILE;
constexpr int FN_OFF_SFT = FN_OFF_SFW + FN_STAGES * F4_SF;
constexpr int FN_SMEM = FN_OFF_SFT + FN_STAGES * F4_SF + 1024;
constexpr uint32_t FN_TMEM_SF = 256;  // after two accumulators of 128 columns: 16 columns per stage
static_assert(FN_TMEM_SF + 16 * FN_STAGES <= 512, "tensor-memory columns");
static_assert(FN_SMEM <= 214 * 1024, "shared memory per CTA, with the table of the groups");

constexpr int FN_MAX_G = 1024;  // groups whose first tiles are kept in shared memory

__device__ __forceinline__ void mma_f4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}

__device__ __forceinline__ void tmem_cp_sf(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

struct TokenTile {
    int64_t row0;   // first row
    int mt;         // its 128-row scale tile (padded order)
    int valid;      // rows of the group from row0 on, at most 128
    int g;
};

// Per group: the 128-row tiles of the groups before it, and its first row.
struct GroupTable {
    int tile[FN_MAX_G + 1];
    int start[FN_MAX_G + 1];
};

// A warp: the table of G <= FN_MAX_G groups over M rows; returns the number of tiles.
__device__ int fill_table(const int32_t* __restrict__ offs, int G, int64_t M, GroupTable* tab) {
    const int lane = threadIdx.x & 31;
    int run = 0, tiles = 0;
    for (int h0 = 0; h0 < G; h0 += 32) {
        const int h = h0 + lane;
        int e = h < G ? (int)min((int64_t)max(offs[h], 0), M) : 0;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int o = __shfl_up_sync(FULL_MASK, e, sh);
            if (lane >= sh) e = max(e, o);
        }
        e = max(e, run);
        const int up = __shfl_up_sync(FULL_MASK, e, 1);
        const int start = lane == 0 ? run : up;
        const int n = h < G ? e - start : 0;
        const int nt = (n + 127) / 128;
        int it = nt;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int ot = __shfl_up_sync(FULL_MASK, it, sh);
            if (lane >= sh) it += ot;
        }
        if (h < G) {
            tab->tile[h] = tiles + it - nt;
            tab->start[h] = start;
            if (h == G - 1) {
                tab->tile[G] = tiles + it;
                tab->start[G] = e;
            }
        }
        tiles += __shfl_sync(FULL_MASK, it, 31);
        run = __shfl_sync(FULL_MASK, e, 31);
    }
    return tiles;
}

__device__ __forceinline__ TokenTile find_tile(const GroupTable& tab, int G, int t) {
    int lo = 0, hi = G;  // tile[lo] <= t < tile[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.tile[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    TokenTile r;
    const int j = t - tab.tile[lo];
    r.g = lo;
    r.row0 = tab.start[lo] + (int64_t)j * 128;
    r.valid = min(128, (int)(tab.start[lo + 1] - r.row0));
    r.mt = t;
    return r;
}

__global__ void __launch_bounds__(192, 1) f4_gemm_narrow_kernel(
    const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap tmap,
    const __grid_constant__ CUtensorMap tmap8,
    const __grid_constant__ CUtensorMap sfwmap, const __grid_constant__ CUtensorMap sftmap,
    const int32_t* __restrict__ offs, int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* __restrict__ out) {
    constexpr int S = FN_STAGES;
    extern __shared__ uint8_t dyn_smem[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[S], empty[S], acc_full[2], acc_empty[2], drained;
    __shared__ GroupTable tab;
    __shared__ uint32_t tmem_base_s;
    __shared__ int n_tiles_s, abort_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n_w = N / F4_ROWS;  // weight tiles of a group
    const int64_t k_blocks = (K + F4_BK - 1) / F4_BK;
    const int64_t col_tiles = K / 128;

    if (warp == 0) {
        const int n = fill_table(offs, G, M, &tab);
        if (lane == 0) {
            n_tiles_s = n;
            abort_s = 0;
            for (int s = 0; s < S; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            for (int s = 0; s < 2; ++s) {
                mbar_init(&acc_full[s], 1);
                mbar_init(&acc_empty[s], 4);
            }
            mbar_init(&drained, 1);
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_addr(&tmem_base_s))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int64_t n_work = n_tiles_s * n_w;

    uint32_t it_prod = 0;
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
            bool stop = false;
            for (int64_t w = blockIdx.x; w < n_work && !stop; w += gridDim.x) {
                const TokenTile tt = find_tile(tab, G, (int)(w / n_w));
                const int64_t n0 = (w % n_w) * F4_ROWS;
                // up to 24 tokens in pieces of 8 rows, more in pieces of 32
                const int box = tt.valid <= 24 ? 8 : 32;
                const CUtensorMap* tm = tt.valid <= 24 ? &tmap8 : &tmap;
                const int pieces = (tt.valid + box - 1) / box;
                const uint32_t tx = F4_TILE + 2 * F4_SF + (uint32_t)(pieces * box * F4_BKB);
                const int64_t sft_row = 2 * (int64_t)tt.mt * col_tiles;
                const int64_t sfw_row = 2 * ((int64_t)tt.g * n_w + n0 / 128) * col_tiles;
                const int w_row = (int)((int64_t)tt.g * N + n0);
                for (int64_t kb = 0; kb < k_blocks; ++kb, ++it_prod) {
                    const int s = (int)(it_prod % S);
                    const uint32_t r = it_prod / S;
                    if (!mbar_wait_bounded(&empty[s], (r & 1) ^ 1, GG_WAIT_NS) || *(volatile int*)&abort_s) {
                        atomicExch(&abort_s, 1);
                        stop = true;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[s], tx);
                    tma_load_2d(sm + s * F4_TILE, &wmap, (int)(kb * F4_BKB), w_row, &full[s], once);
                    tma_load_2d(sm + FN_OFF_SFW + s * F4_SF, &sfwmap, 0, (int)(sfw_row + 4 * kb), &full[s], once);
                    for (int p = 0; p < pieces; ++p)
                        tma_load_2d(sm + FN_OFF_T + s * F4_TILE + p * box * F4_BKB, tm, (int)(kb * F4_BKB),
                                    (int)tt.row0 + p * box, &full[s], keep);
                    tma_load_2d(sm + FN_OFF_SFT + s * F4_SF, &sftmap, 0, (int)(sft_row + 4 * kb), &full[s], keep);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t it = 0;
            int64_t i = 0;
            for (int64_t w = blockIdx.x; w < n_work; w += gridDim.x, ++i) {
                const uint32_t cols = (uint32_t)(find_tile(tab, G, (int)(w / n_w)).valid + 31) / 32 * 32;
                const int buf = (int)(i & 1);
                if (i > 1 && !mbar_wait_bounded(&acc_empty[buf], (uint32_t)((i / 2 - 1) & 1), GG_WAIT_NS)) {
                    atomicExch(&abort_s, 1);
                    break;
                }
                tc_fence_after();
                bool ok = true;
                for (int64_t kb = 0; kb < k_blocks; ++kb, ++it) {
                    const int s = (int)(it % S);
                    if (!mbar_wait_bounded(&full[s], (it / S) & 1, GG_WAIT_NS) || *(volatile int*)&abort_s) {
                        atomicExch(&abort_s, 1);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t t_w = tmem + FN_TMEM_SF + 16 * s, t_t = t_w + 8;
                    const uint8_t* sfw = sm + FN_OFF_SFW + s * F4_SF;
                    const uint8_t* sft = sm + FN_OFF_SFT + s * F4_SF;
                    tmem_cp_sf(t_w, desc_sf(sfw));
                    tmem_cp_sf(t_w + 4, desc_sf(sfw + 512));
                    tmem_cp_sf(t_t, desc_sf(sft));
                    tmem_cp_sf(t_t + 4, desc_sf(sft + 512));
                    const uint64_t a0 = desc_sw128(sm + s * F4_TILE), b0 = desc_sw128(sm + FN_OFF_T + s * F4_TILE);
                    const uint32_t nk = K - kb * F4_BK >= F4_BK ? 4 : 2;
                    for (uint32_t k = 0; k < nk; ++k) {
                        const uint32_t id = 2 * (k & 1), t = k >> 1;
                        mma_f4(tmem + buf * 128, a0 + 2 * k, b0 + 2 * k, idesc_f4<128>(cols, id),
                               (t_w + 4 * t) | id << 30, (t_t + 4 * t) | id << 30, (kb > 0 || k > 0) ? 1u : 0u);
                    }
                    mma_commit(&empty[s]);
                }
                if (!ok) break;
                mma_commit(&acc_full[buf]);
            }
            mma_commit(&drained);
            if (!mbar_wait_bounded(&drained, 0, GG_DRAIN_NS)) atomicExch(&abort_s, 1);
        }
        __syncwarp();
    } else {
        // ---- epilogue: lane = weight row (output column), register = token
        const int quarter = warp & 3;
        int64_t i = 0;
        for (int64_t w = blockIdx.x; w < n_work; w += gridDim.x, ++i) {
            const TokenTile tt = find_tile(tab, G, (int)(w / n_w));
            const int64_t n0 = (w % n_w) * F4_ROWS;
            const int buf = (int)(i & 1);
            const bool done = mbar_wait_bounded(&acc_full[buf], (uint32_t)((i / 2) & 1), GG_WAIT_NS);
            if (!done) atomicExch(&abort_s, 1);
            if (__any_sync(FULL_MASK, !done) || *(volatile int*)&abort_s) break;
            tc_fence_after();
            uint16_t* o = out + tt.row0 * N + n0 + 32 * quarter + lane;
            for (int c0 = 0; c0 < tt.valid; c0 += 32) {
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(buf * 128 + c0), v);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c0 + j < tt.valid) o[(int64_t)(c0 + j) * N] = (uint16_t)cvt_bf16x2(__uint_as_float(v[j]), 0.0f);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
    }

    // ---- leaving: every copy has landed before the CTA's shared memory goes
    if (warp == 0 && lane == 0)
        for (uint32_t i = it_prod > (uint32_t)S ? it_prod - S : 0u; i < it_prod; ++i)
            if (!mbar_wait_bounded(&full[i % S], (i / S) & 1, GG_DRAIN_NS)) atomicExch(&abort_s, 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (abort_s && tid == 0) atomicAdd(&g_f4_gemm_timeouts, 1u);
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ---- host side -----------------------------------------------------------------------------------

bool use_narrow(int64_t M, int32_t G) { return G <= FN_MAX_G && M <= 128 * (int64_t)G; }

struct Maps {
    CUtensorMap a, b, sfa, sfb;
};

// Row boxes of `a_rows` tokens and `b_rows` weights; two scale tiles (4 rows of 256 bytes).
bool encode_maps(Maps* m, const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb, int64_t G,
                 int64_t M, int64_t N, int64_t K, int64_t sfa_rows, int64_t sfb_rows, int a_rows, int b_rows) {
    std::memset(m, 0, sizeof(*m));
    return encode_u8_tile_map_sw128(&m->a, qa, (uint64_t)K / 2, (uint64_t)M, F4_BKB, a_rows) &&
           encode_u8_tile_map_sw128(&m->b, qb, (uint64_t)K / 2, (uint64_t)G * N, F4_BKB, b_rows) &&
           encode_u8_map_plain(&m->sfa, sfa, 256, (uint64_t)sfa_rows, 256, 4) &&
           encode_u8_map_plain(&m->sfb, sfb, 256, (uint64_t)sfb_rows, 256, 4);
}

cudaError_t launch_narrow(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb,
                          const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, int64_t sfa_rows,
                          int64_t sfb_rows, uint16_t* out, cudaStream_t stream) {
    Maps m;
    CUtensorMap a8;
    std::memset(&a8, 0, sizeof(a8));
    if (!encode_maps(&m, qa, sfa, qb, sfb, G, M, N, K, sfa_rows, sfb_rows, 32, F4_ROWS) ||
        !encode_u8_tile_map_sw128(&a8, qa, (uint64_t)K / 2, (uint64_t)M, F4_BKB, 8))
        return cudaErrorInvalidValue;
    const cudaError_t e =
        cudaFuncSetAttribute(f4_gemm_narrow_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FN_SMEM);
    if (e != cudaSuccess) return e;
    const int64_t units = std::min((M + 127 * (int64_t)G) / 128, M) * (N / F4_ROWS);  // an upper bound
    const unsigned grid = (unsigned)std::min<int64_t>(units, sm_count());
    f4_gemm_narrow_kernel<<<grid, 192, FN_SMEM, stream>>>(m.b, m.a, a8, m.sfb, m.sfa, offs, G, M, N, K, out);
    return cudaGetLastError();
}

}  // namespace

unsigned int read_f4_gemm_timeouts() {
    unsigned int n = 0;
    if (cudaMemcpyFromSymbol(&n, g_f4_gemm_timeouts, sizeof(n)) != cudaSuccess) return 0xFFFFFFFFu;
    return n;
}

cudaError_t launch_mxfp4_grouped_gemm(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb,
                                      const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, uint16_t* out,
                                      cudaStream_t stream) {
    const int64_t m_tiles = (M + (int64_t)(F4_ROWS - 1) * G) / F4_ROWS;  // bound on the groups' padded tiles
    if (m_tiles <= 0 || N == 0 || K == 0) return cudaSuccess;
    const int64_t col_tiles = K / 128;
    const int64_t sfa_rows = 2 * m_tiles * col_tiles, sfb_rows = 2 * (int64_t)G * (N / 128) * col_tiles;
    if (M + 256 > 0x7FFFFFFFLL || (int64_t)G * N > 0x7FFFFFFFLL || sfa_rows + 4 > 0x7FFFFFFFLL ||
        sfb_rows + 4 > 0x7FFFFFFFLL || K / 2 > 0x7FFFFF00LL)
        return cudaErrorInvalidConfiguration;
    if (use_narrow(M, G))
        return launch_narrow(qa, sfa, qb, sfb, offs, G, M, N, K, sfa_rows, sfb_rows, out, stream);
    Maps m;
    if (!encode_maps(&m, qa, sfa, qb, sfb, G, M, N, K, sfa_rows, sfb_rows, F4_ROWS, F4_ROWS))
        return cudaErrorInvalidValue;
    const cudaError_t e =
        cudaFuncSetAttribute(f4_gemm_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FW_SMEM);
    if (e != cudaSuccess) return e;
    const int64_t units = (m_tiles + G) / 2 * (N / FW_BN);
    const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(units, sm_count() / 2));
    f4_gemm_wide_kernel<<<(unsigned)(2 * pairs), 192, FW_SMEM, stream>>>(m.a, m.b, m.sfa, m.sfb, offs, G, M, N, K,
                                                                         out);
    return cudaGetLastError();
}

}  // namespace mxq
