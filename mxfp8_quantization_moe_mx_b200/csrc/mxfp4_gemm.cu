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
// Both are persistent, with a producer warp (TMA), an MMA warp, four epilogue warps, and every
// wait bounded as in the MXFP8 kernel (mxq_wait_timeouts counts CTAs that gave up).

#include <algorithm>
#include <cstring>

#include "dependent.cuh"
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
// Tensor memory: two accumulators of 256 columns that share 64, and two slots of 8 + 16
// scale columns.  A unit's epilogue reads the shared columns first, so the next unit's MMAs
// wait for a quarter of it.
constexpr uint32_t FW_ACC1 = 192;
constexpr uint32_t FW_SHARED = 64;
constexpr uint32_t FW_TMEM_SF = 448;
static_assert(FW_ACC1 + FW_SHARED == FW_BN && FW_ACC1 + FW_BN == FW_TMEM_SF && FW_TMEM_SF + 2 * 24 <= 512,
              "tensor-memory columns");
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

// One lane of the (converged) warp.  The producer and MMA warps walk their units with all
// lanes and let an elected lane issue: descriptors, addresses and loop state then stay in
// uniform registers, which the TMA and MMA instructions take them from.  Issued by one lane
// of a diverged warp instead, an MMA took about twice its own time to issue (20 K blocks of
// a 256 x 256 unit: 0.71 us each against 0.56).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A wait of the whole warp with one outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(FULL_MASK, mbar_wait_bounded(bar, parity, GG_WAIT_NS));
}

// Instruction descriptor of kind::mxf4: E2M1 A and B, E8M0 scales, an M x N tile; `id` the
// first of the two scale bytes (0 or 2) of the A and B scale columns.
template <int M>
__device__ __forceinline__ uint32_t idesc_f4(uint32_t n, uint32_t id) {
    constexpr uint32_t base = 1u << 7 | 1u << 10 | 1u << 23 | (uint32_t)(M >> 4) << 24;
    return base | (n >> 3) << 17 | id << 4 | id << 29;
}

// 32 consecutive fp32 columns of this warp's 32 tensor-memory lanes into v[0..31], which hold
// them once tmem_wait_ld has returned.
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

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
    const int64_t col_tiles = K / 128;

    if (warp == 0 && lane == 0) {
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
    // The operands and offsets are the work of earlier kernels.  Tensor memory is taken after
    // they have ended and before later ones may come: a kernel that waits for another holds
    // none of it.
    grid_depend_wait();
    if (warp == 1) tmem_alloc_pair(&tmem_base_s, 512);
    if (warp == 0) {
        PairTile pt;
        int64_t total;
        gg_find_pair(offs, G, M, -1, &pt, &total);
        if (lane == 0) n_work_s = total * n_tiles_n;
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers are initialised before either signals the other's
    tc_fence_after();
    grid_release();
    const uint32_t tmem = tmem_base_s;
    const int64_t n_work = n_work_s;
    const uint32_t full0 = cluster_map(&full[0], 0);  // the first CTA's `full` ring (8 bytes apart)
    const uint32_t acc_empty0 = cluster_map(&acc_empty, 0);

    const int k_full = (int)(K / F4_BK), k_half = (int)(K % F4_BK != 0);
    uint32_t it_prod = 0;
    if (warp == 0) {
        // ---- producer (both CTAs)
        const uint64_t pol = l2_policy_evict_last();
        const bool el = elect_one();
        uint32_t s = 0, ph = 1;
        bool ok = true;
        for (int64_t w = cl; w < n_work && ok; w += n_cl) {
            const int64_t p = w / n_tiles_n, n0 = (w % n_tiles_n) * FW_BN;
            PairTile pt;
            gg_find_pair(offs, G, M, p, &pt, nullptr);
            const int my_row = (int)(pt.row0 + (int64_t)rank * F4_ROWS);
            const int64_t my_mt = (rank == 1 && pt.valid1 > 0) ? pt.mt0 + 1 : pt.mt0;  // filler: any real tile
            int sfa_row = (int)(2 * my_mt * col_tiles);
            int sfb_row = (int)(2 * ((int64_t)pt.g * (N / 128) + n0 / 128) * col_tiles);
            const int sfb_half = (int)(2 * col_tiles);
            const int b_row = (int)((int64_t)pt.g * N + n0 + (int64_t)rank * (FW_BN / 2));
            for (int kb = 0; kb < k_full + k_half; ++kb, ++it_prod, sfa_row += 4, sfb_row += 4) {
                if (!warp_wait(&empty[s], ph) || *(volatile int*)&abort_s) {
                    ok = false;
                    break;
                }
                if (el) {
                    if (first) mbar_arrive_expect_tx(&full[s], 2 * FW_CTA_TX);
                    const uint32_t bar = full0 + 8u * s;
                    tma_load_2d_pair(sm + s * F4_TILE, &amap, kb * F4_BKB, my_row, bar, pol);
                    tma_load_2d_pair(sm + FW_OFF_B + s * F4_TILE, &bmap, kb * F4_BKB, b_row, bar, pol);
                    tma_load_2d_pair(sm + FW_OFF_SFA + s * F4_SF, &sfamap, 0, sfa_row, bar, pol);
                    tma_load_2d_pair(sm + FW_OFF_SFB + s * 2 * F4_SF, &sfbmap, 0, sfb_row, bar, pol);
                    tma_load_2d_pair(sm + FW_OFF_SFB + s * 2 * F4_SF + F4_SF, &sfbmap, 0, sfb_row + sfb_half, bar,
                                     pol);
                }
                if (++s == FW_STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok && el) atomicExch(&abort_s, 1);
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer (the first CTA)
        if (first) {
            const bool el = elect_one();
            const uint64_t a_base = desc_sw128(sm), b_base = desc_sw128(sm + FW_OFF_B);
            const uint64_t sfa_base = desc_sf(sm + FW_OFF_SFA), sfb_base = desc_sf(sm + FW_OFF_SFB);
            constexpr uint32_t T = F4_TILE / 16, SF = F4_SF / 16;  // descriptor units of 16 bytes
            uint32_t s = 0, ph = 0, slot = 0, unit = 0;
            bool ok = true;
            for (int64_t w = cl; w < n_work; w += n_cl, ++unit) {
                if (unit > 0 && !warp_wait(&acc_empty, (unit - 1) & 1)) ok = false;
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + (unit & 1 ? FW_ACC1 : 0);
                for (int kb = 0; kb < k_full + k_half; ++kb) {
                    if (!warp_wait(&full[s], ph)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (el) {
                        // scale columns: A [scale tile][4], B [scale tile][column half][4]; copies
                        // and MMAs of one thread run in order, so two slots are enough
                        const uint32_t t_a = tmem + FW_TMEM_SF + 24 * slot, t_b = t_a + 8;
                        const uint64_t sfa = sfa_base + s * SF, sfb = sfb_base + s * 2 * SF;
                        const uint64_t a0 = a_base + s * T, b0 = b_base + s * T;
                        tmem_cp_sf_pair(t_a, sfa);
                        tmem_cp_sf_pair(t_b, sfb);
                        tmem_cp_sf_pair(t_b + 4, sfb + SF);
                        tmem_cp_sf_pair(t_a + 4, sfa + SF / 2);
                        tmem_cp_sf_pair(t_b + 8, sfb + SF / 2);
                        tmem_cp_sf_pair(t_b + 12, sfb + SF + SF / 2);
                        // K = 64 per MMA: 32 bytes further along the swizzled rows
                        constexpr uint32_t HI = 2u << 30;  // the upper two scale bytes of a column
                        mma_f4_pair(acc, a0, b0, idesc_f4<256>(FW_BN, 0), t_a, t_b, kb > 0);
                        mma_f4_pair(acc, a0 + 2, b0 + 2, idesc_f4<256>(FW_BN, 2), t_a | HI, t_b | HI, 1);
                        if (kb < k_full) {
                            mma_f4_pair(acc, a0 + 4, b0 + 4, idesc_f4<256>(FW_BN, 0), t_a + 4, t_b + 8, 1);
                            mma_f4_pair(acc, a0 + 6, b0 + 6, idesc_f4<256>(FW_BN, 2), (t_a + 4) | HI, (t_b + 8) | HI,
                                        1);
                        }
                        mma_commit_both(&empty[s]);  // the stage is free in both CTAs once these have read it
                        if (kb == k_full + k_half - 1) mma_commit_both(&acc_full);
                    }
                    __syncwarp();
                    slot ^= 1;
                    if (++s == FW_STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                if (!ok) break;  // a partial accumulator is never handed to the epilogues
            }
            // every tcgen05 operation issued above (and its arrivals) is done before the pair
            // frees tensor memory or leaves
            if (el) {
                if (!ok) atomicExch(&abort_s, 1);
                mma_commit_own(&drained);
                if (!mbar_wait_bounded(&drained, 0, GG_DRAIN_NS)) atomicExch(&abort_s, 1);
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue (both CTAs): warp w reads accumulator lanes (rows) 32 (w % 4) .. + 31
        const int quarter = warp & 3;
        const int r = 32 * quarter + lane;
        uint32_t unit = 0;
        for (int64_t w = cl; w < n_work; w += n_cl, ++unit) {
            const int64_t p = w / n_tiles_n, n0 = (w % n_tiles_n) * FW_BN;
            PairTile pt;
            gg_find_pair(offs, G, M, p, &pt, nullptr);
            const bool done = mbar_wait_bounded(&acc_full, unit & 1, GG_WAIT_NS);
            if (!done) atomicExch(&abort_s, 1);
            if (__any_sync(FULL_MASK, !done) || *(volatile int*)&abort_s) break;
            tc_fence_after();
            const uint32_t acc = tmem + (unit & 1 ? FW_ACC1 : 0) + ((uint32_t)(32 * quarter) << 16);
            // the shared columns first: the last of the even units' accumulator, the first of
            // the odd units'
            const int c_first = unit & 1 ? 0 : FW_BN - (int)FW_SHARED;
            const bool live = r < (rank == 0 ? pt.valid0 : pt.valid1);
            uint16_t* orow = out + (pt.row0 + (int64_t)rank * F4_ROWS + r) * N + n0;
#pragma unroll 1
            for (int i = 0; i < FW_BN / 64; ++i) {
                const int c0 = (c_first + 64 * i) & (FW_BN - 1);
                uint32_t v[64];
                tmem_ld32_nowait(acc + (uint32_t)c0, v);
                tmem_ld32_nowait(acc + (uint32_t)c0 + 32, v + 32);
                tmem_wait_ld();
                if (i == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(acc_empty0);  // this warp's shared columns are read
                }
                if (live) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        uint32_t o[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            o[j] = cvt_bf16x2(__uint_as_float(v[8 * q + 2 * j]), __uint_as_float(v[8 * q + 2 * j + 1]));
                        *reinterpret_cast<uint4*>(orow + c0 + 8 * q) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
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
constexpr uint32_t FN_TMEM_SF = 256;  // after two accumulators of 128 columns: two slots of 16 columns
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
    const int64_t col_tiles = K / 128;

    if (warp == 0 && lane == 0) {
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
    grid_depend_wait();  // then tensor memory, as in the wide kernel
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_addr(&tmem_base_s))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 0) {
        const int n = fill_table(offs, G, M, &tab);
        if (lane == 0) n_tiles_s = n;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_release();
    const uint32_t tmem = tmem_base_s;
    const int64_t n_work = n_tiles_s * n_w;

    const int k_full = (int)(K / F4_BK), k_half = (int)(K % F4_BK != 0);
    uint32_t it_prod = 0;
    if (warp == 0) {
        const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
        const bool el = elect_one();
        uint32_t s = 0, ph = 1;
        bool ok = true;
        for (int64_t w = blockIdx.x; w < n_work && ok; w += gridDim.x) {
            const TokenTile tt = find_tile(tab, G, (int)(w / n_w));
            const int64_t n0 = (w % n_w) * F4_ROWS;
            // up to 24 tokens in pieces of 8 rows, more in pieces of 32
            const int box = tt.valid <= 24 ? 8 : 32;
            const CUtensorMap* tm = tt.valid <= 24 ? &tmap8 : &tmap;
            const int pieces = (tt.valid + box - 1) / box;
            const uint32_t tx = F4_TILE + 2 * F4_SF + (uint32_t)(pieces * box * F4_BKB);
            int sft_row = (int)(2 * (int64_t)tt.mt * col_tiles);
            int sfw_row = (int)(2 * ((int64_t)tt.g * n_w + n0 / 128) * col_tiles);
            const int w_row = (int)((int64_t)tt.g * N + n0), t_row = (int)tt.row0;
            for (int kb = 0; kb < k_full + k_half; ++kb, ++it_prod, sft_row += 4, sfw_row += 4) {
                if (!warp_wait(&empty[s], ph) || *(volatile int*)&abort_s) {
                    ok = false;
                    break;
                }
                if (el) {
                    mbar_arrive_expect_tx(&full[s], tx);
                    tma_load_2d(sm + s * F4_TILE, &wmap, kb * F4_BKB, w_row, &full[s], once);
                    tma_load_2d(sm + FN_OFF_SFW + s * F4_SF, &sfwmap, 0, sfw_row, &full[s], once);
                    for (int p = 0; p < pieces; ++p)
                        tma_load_2d(sm + FN_OFF_T + s * F4_TILE + p * box * F4_BKB, tm, kb * F4_BKB, t_row + p * box,
                                    &full[s], keep);
                    tma_load_2d(sm + FN_OFF_SFT + s * F4_SF, &sftmap, 0, sft_row, &full[s], keep);
                }
                if (++s == S) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok && el) atomicExch(&abort_s, 1);
        __syncwarp();
    } else if (warp == 1) {
        const bool el = elect_one();
        const uint64_t w_base = desc_sw128(sm), t_base = desc_sw128(sm + FN_OFF_T);
        const uint64_t sfw_base = desc_sf(sm + FN_OFF_SFW), sft_base = desc_sf(sm + FN_OFF_SFT);
        constexpr uint32_t T = F4_TILE / 16, SF = F4_SF / 16;  // descriptor units of 16 bytes
        uint32_t s = 0, ph = 0, slot = 0, unit = 0;
        bool ok = true;
        for (int64_t w = blockIdx.x; w < n_work; w += gridDim.x, ++unit) {
            const uint32_t cols = (uint32_t)(find_tile(tab, G, (int)(w / n_w)).valid + 31) / 32 * 32;
            const uint32_t buf = unit & 1;
            if (unit > 1 && !warp_wait(&acc_empty[buf], (unit / 2 - 1) & 1)) ok = false;
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * 128;
            const uint32_t id0 = idesc_f4<128>(cols, 0), id2 = idesc_f4<128>(cols, 2);
            for (int kb = 0; kb < k_full + k_half; ++kb) {
                if (!warp_wait(&full[s], ph)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (el) {
                    const uint32_t t_w = tmem + FN_TMEM_SF + 16 * slot, t_t = t_w + 8;
                    const uint64_t sfw = sfw_base + s * SF, sft = sft_base + s * SF;
                    const uint64_t a0 = w_base + s * T, b0 = t_base + s * T;
                    tmem_cp_sf(t_w, sfw);
                    tmem_cp_sf(t_t, sft);
                    tmem_cp_sf(t_w + 4, sfw + SF / 2);
                    tmem_cp_sf(t_t + 4, sft + SF / 2);
                    constexpr uint32_t HI = 2u << 30;
                    mma_f4(acc, a0, b0, id0, t_w, t_t, kb > 0);
                    mma_f4(acc, a0 + 2, b0 + 2, id2, t_w | HI, t_t | HI, 1);
                    if (kb < k_full) {
                        mma_f4(acc, a0 + 4, b0 + 4, id0, t_w + 4, t_t + 4, 1);
                        mma_f4(acc, a0 + 6, b0 + 6, id2, (t_w + 4) | HI, (t_t + 4) | HI, 1);
                    }
                    mma_commit(&empty[s]);
                    if (kb == k_full + k_half - 1) mma_commit(&acc_full[buf]);
                }
                __syncwarp();
                slot ^= 1;
                if (++s == S) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (!ok) break;
        }
        if (el) {
            if (!ok) atomicExch(&abort_s, 1);
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

// The narrow kernel for groups of up to 112 rows on average, which then mostly fill one token
// tile, and for products so small that the wide units would leave SMs idle and the narrow
// ones fit in one wave.  Measured, narrow / wide: 16 matrices of 8192 x 5120 with 24 rows
// 64 / 96 us, 512 rows 66 / 84, 1792 rows 78 / 89, 3000 rows 119 / 92, 16411 rows 471 / 296;
// one matrix of 8192 x 5120 with 256 rows 16 / 20, 512 rows 25 / 20; one of 2048 x 2048 with
// 1024 rows 12 / 14.
bool use_narrow(int64_t M, int32_t G, int64_t N) {
    const int64_t units = std::min((M + 127 * (int64_t)G) / 128, M) * (N / F4_ROWS);  // an upper bound
    return G <= FN_MAX_G && (M <= 112 * (int64_t)G || units <= sm_count());
}

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
    return launch_dependent(f4_gemm_narrow_kernel, grid, 192, FN_SMEM, stream, m.b, m.a, a8, m.sfb, m.sfa, offs, G, M,
                            N, K, out);
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
    if (use_narrow(M, G, N))
        return launch_narrow(qa, sfa, qb, sfb, offs, G, M, N, K, sfa_rows, sfb_rows, out, stream);
    Maps m;
    if (!encode_maps(&m, qa, sfa, qb, sfb, G, M, N, K, sfa_rows, sfb_rows, F4_ROWS, F4_ROWS))
        return cudaErrorInvalidValue;
    const cudaError_t e =
        cudaFuncSetAttribute(f4_gemm_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FW_SMEM);
    if (e != cudaSuccess) return e;
    const int64_t units = (m_tiles + G) / 2 * (N / FW_BN);
    const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(units, sm_count() / 2));
    return launch_dependent(f4_gemm_wide_kernel, (unsigned)(2 * pairs), 192, FW_SMEM, stream, m.a, m.b, m.sfa, m.sfb,
                            offs, G, M, N, K, out);
}

}  // namespace mxq
