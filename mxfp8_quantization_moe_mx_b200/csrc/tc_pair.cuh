// tc_pair.cuh -- tcgen05 (5th-generation tensor core) wrappers and the unit walk shared by
// the block-scaled grouped GEMMs.
#pragma once

#include "mxq_device.cuh"

namespace mxq {

constexpr int GG_BM = 128;                             // rows per CTA (the paired MMA: 256)
constexpr uint64_t GG_WAIT_NS = 2000000000ull, GG_DRAIN_NS = 20000000000ull;

// ---- tcgen05 / cluster wrappers (paired forms) -----------------------------------------------

// TMA 2-D tile load into this CTA's shared memory that completes on an mbarrier of either
// CTA of the pair (`bar` a cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* tmap, int x, int y, uint32_t bar,
                                                 uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_addr(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(bar), "l"(pol)
        : "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Count `bytes` as arrived on the current phase's transaction count (no arrival).
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Whole-cluster barrier with release / acquire (every thread of both CTAs).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 bytes
// apart (rows of 128 bytes), Blackwell descriptor version 1.
__device__ __forceinline__ uint64_t desc_sw128(const void* p) {
    const uint64_t a = (smem_addr(p) & 0x3FFFFu) >> 4;
    return a | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Descriptor of a dense 32-row x 16-byte block (a 512-byte scale tile): no swizzle,
// 8-row core matrices 128 bytes apart.
__device__ __forceinline__ uint64_t desc_sf(const void* p) {
    const uint64_t a = (smem_addr(p) & 0x3FFFFu) >> 4;
    return a | (8ull << 32) | (1ull << 46);
}

// Paired copy: each CTA's 512-byte scale tile at this shared-memory offset into 4 columns
// of its own tensor memory (copied to all four lane quarters).
__device__ __forceinline__ void tmem_cp_sf_pair(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Arrives (once) on the mbarrier at this shared-memory offset in both CTAs of the pair
// when every tcgen05 operation this thread issued before it has completed.
__device__ __forceinline__ void mma_commit_both(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// ... on this CTA's mbarrier only.
__device__ __forceinline__ void mma_commit_own(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// 32 consecutive fp32 columns of this warp's 32 tensor-memory lanes (one row per lane).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---- unit walk ------------------------------------------------------------------------------

struct PairTile {
    int64_t row0;    // first row of the unit (the first CTA's rows; the second's start 128 later)
    int64_t valid0;  // rows of the group in the first CTA's 128 (>= 1)
    int64_t valid1;  // ... in the second CTA's 128 (<= 0: none)
    int64_t mt0;     // padded M-tile index of the first CTA's rows (its scale tile)
    int g;           // the group (expert)
};

// Run by a whole warp: M pair `pair` -- the groups' padded M tiles taken two at a time
// within each group, groups in order -- returned to every lane.  With pair < 0 only the
// number of pairs is computed (into *total).
static __device__ void gg_find_pair(const int32_t* __restrict__ offs, int32_t G, int64_t M, int64_t pair, PairTile* pt,
                                    int64_t* total) {
    const int lane = threadIdx.x & 31;
    int run = 0;
    int64_t tiles_before = 0, pairs_before = 0;
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
        const int64_t end = min((int64_t)e, M), start = min((int64_t)prev_e, M);
        const int64_t n_tiles = h < G ? (end - start + GG_BM - 1) / GG_BM : 0;
        const int64_t n_pairs = (n_tiles + 1) / 2;
        int64_t inc_t = n_tiles, inc_p = n_pairs;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int64_t ot = __shfl_up_sync(FULL_MASK, inc_t, sh);
            const int64_t op = __shfl_up_sync(FULL_MASK, inc_p, sh);
            if (lane >= sh) {
                inc_t += ot;
                inc_p += op;
            }
        }
        const int64_t first_t = tiles_before + inc_t - n_tiles, first_p = pairs_before + inc_p - n_pairs;
        const bool mine = pair >= 0 && h < G && pair >= first_p && pair < first_p + n_pairs;
        const unsigned who = __ballot_sync(FULL_MASK, mine);
        if (who) {
            const int src = __ffs(who) - 1;
            const int64_t j = 2 * (pair - first_p);
            const int64_t my_r0 = start + j * GG_BM;
            pt->row0 = __shfl_sync(FULL_MASK, my_r0, src);
            pt->valid0 = __shfl_sync(FULL_MASK, min((int64_t)GG_BM, end - my_r0), src);
            pt->valid1 = __shfl_sync(FULL_MASK, min((int64_t)GG_BM, end - my_r0 - GG_BM), src);
            pt->mt0 = __shfl_sync(FULL_MASK, first_t + j, src);
            pt->g = __shfl_sync(FULL_MASK, h, src);
            found = true;
        }
        tiles_before += __shfl_sync(FULL_MASK, inc_t, 31);
        pairs_before += __shfl_sync(FULL_MASK, inc_p, 31);
        run = __shfl_sync(FULL_MASK, e, 31);
    }
    if (total) *total = pairs_before;
}

}  // namespace mxq
