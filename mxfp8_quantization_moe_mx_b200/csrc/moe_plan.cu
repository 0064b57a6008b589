// moe_plan.cu -- from the experts of each token to the rows of the grouped products
// (sm_100a).
//
// ids (n = T * k values in 0..E-1, or out of range: routed nowhere) -> a stable sort by
// expert: row r of the grouped operand holds slot src[r] (token src[r] / k), group e is
// rows [offs[e-1], offs[e]), rows[slot] is the slot's row or -1.  A counting sort:
//   one CTA (n <= PL_ONE) keeps everything in shared memory: every warp counts its run of
//   consecutive slots by expert, the counts become starts, every slot takes its row.
//   Else a CTA per chunk of PL_CHUNK slots in three launches, each dependent on the one
//   before: count writes the chunk's count of every expert to the workspace, [E][chunks];
//   scan, a warp per expert, turns them into the slots of that expert in earlier chunks,
//   and its total; place proceeds as the one CTA does, from those.
// Ranks among 32 neighbouring slots come from a match of equal ids, so the order is that of
// the slots and no atomic decides it.
//
// The bytes (12 per slot) are few: what it costs is the launches and the latency of each
// step.  524288 slots over 256 experts: see the launcher.

#include <algorithm>

#include "mxq_device.cuh"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int PL_CHUNK = 2048, PL_CHUNK_WARPS = 8;  // 256 slots per warp
constexpr int PL_ONE = 16384, PL_ONE_WARPS = 32;    // at most 512 slots per warp

// Slot `at`'s expert, -1 if it has none.
__device__ __forceinline__ int slot_id(const int32_t* __restrict__ ids, int64_t at, int64_t end, int E) {
    const int v = at < end ? __ldg(ids + at) : -1;
    return v < 0 || v >= E ? -1 : v;
}

// The warp's slots [first, end) by expert, into cnt[0..E) (shared).
__device__ __forceinline__ void warp_count(const int32_t* __restrict__ ids, int64_t first, int64_t end, int E, int* cnt,
                                           int lane) {
    for (int e = lane; e < E; e += 32) cnt[e] = 0;
    __syncwarp();
#pragma unroll 4
    for (int64_t a = first; a < end; a += 32) {
        const int id = slot_id(ids, a + lane, end, E);
        const unsigned same = __match_any_sync(FULL_MASK, id);
        if (id >= 0 && lane == __ffs(same) - 1) cnt[id] += __popc(same);
        __syncwarp();
    }
}

__global__ void __launch_bounds__(32 * PL_CHUNK_WARPS) plan_count_kernel(const int32_t* __restrict__ ids, int64_t n,
                                                                         int E, int32_t* __restrict__ counts) {
    extern __shared__ int plan_s[];
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = (int64_t)blockIdx.x * PL_CHUNK + warp * (PL_CHUNK / PL_CHUNK_WARPS);
    warp_count(ids, first, min(n, first + PL_CHUNK / PL_CHUNK_WARPS), E, plan_s + warp * E, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 32 * PL_CHUNK_WARPS) {
        int c = 0;
#pragma unroll
        for (int w = 0; w < PL_CHUNK_WARPS; ++w) c += plan_s[w * E + e];
        counts[(int64_t)e * gridDim.x + blockIdx.x] = c;
    }
}

// Row e of counts (one warp each) -> its exclusive prefix sums; totals[e] their sum.
__global__ void __launch_bounds__(128) plan_scan_kernel(int32_t* __restrict__ counts, int chunks, int E,
                                                        int32_t* __restrict__ totals) {
    grid_wait();
    const int lane = threadIdx.x & 31, e = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (e >= E) return;
    int32_t* row = counts + (int64_t)e * chunks;
    int run = 0;
    for (int c0 = 0; c0 < chunks; c0 += 128) {
        int v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + 32 * i + lane;
            v[i] = c < chunks ? row[c] : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + 32 * i + lane;
            int inc = v[i];
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int o = __shfl_up_sync(FULL_MASK, inc, s);
                if (lane >= s) inc += o;
            }
            if (c < chunks) row[c] = run + inc - v[i];
            run += __shfl_sync(FULL_MASK, inc, 31);
        }
    }
    if (lane == 0) totals[e] = run;
}

// WARPS warps take `per` consecutive slots each.  before / totals: NULL for the one CTA
// that has all slots (both come from its own counts).
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) plan_place_kernel(const int32_t* __restrict__ ids, int64_t n, int per,
                                                                int E, const int32_t* __restrict__ before,
                                                                const int32_t* __restrict__ totals,
                                                                int32_t* __restrict__ offs, int32_t* __restrict__ rows,
                                                                int32_t* __restrict__ src) {
    extern __shared__ int plan_s[];  // [WARPS][E] counts, then starts; [E] expert starts
    __shared__ int routed_s;
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* starts = plan_s + WARPS * E;
    const int64_t first = ((int64_t)blockIdx.x * WARPS + warp) * per, end = min(n, first + per);
    int* mine = plan_s + warp * E;
    warp_count(ids, first, end, E, mine, lane);
    __syncthreads();
    // per expert: the warps' counts become starts relative to the expert's; its total
    for (int e = threadIdx.x; e < E; e += 32 * WARPS) {
        int run = before ? before[(int64_t)e * gridDim.x + blockIdx.x] : 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const int v = plan_s[w * E + e];
            plan_s[w * E + e] = run;
            run += v;
        }
        starts[e] = totals ? totals[e] : run;
    }
    __syncthreads();
    if (warp == 0) {  // exclusive prefix sum of the totals
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int v = e < E ? starts[e] : 0;
            int inc = v;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int o = __shfl_up_sync(FULL_MASK, inc, s);
                if (lane >= s) inc += o;
            }
            if (e < E) {
                starts[e] = carry + inc - v;
                if (blockIdx.x == 0) offs[e] = carry + inc;
            }
            carry += __shfl_sync(FULL_MASK, inc, 31);
        }
        if (lane == 0) routed_s = carry;
    }
    __syncthreads();
    const int routed = routed_s;
#pragma unroll 4
    for (int64_t a = first; a < end; a += 32) {
        const int64_t at = a + lane;
        const int id = slot_id(ids, at, end, E);
        const unsigned same = __match_any_sync(FULL_MASK, id);
        int r = -1;
        if (id >= 0) r = starts[id] + mine[id] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
        __syncwarp();
        if (at < end) {
            rows[at] = r;
            if (r >= 0) src[r] = (int32_t)at;
            if (at >= routed) src[at] = -1;  // rows behind the last group
        }
    }
}

int64_t plan_chunks(int64_t n) { return (n + PL_CHUNK - 1) / PL_CHUNK; }

}  // namespace

// The one CTA needs none: its counts never leave it.
int64_t plan_workspace_bytes(int64_t n, int E) { return n <= PL_ONE ? 0 : 4 * (plan_chunks(n) + 1) * E; }

cudaError_t launch_moe_plan(const int32_t* ids, int64_t n, int E, int32_t* offs, int32_t* rows, int32_t* src,
                            int32_t* ws, cudaStream_t stream) {
    if (n <= PL_ONE) {
        // a slot per lane and step, at least one step for each warp
        const size_t smem = (size_t)(PL_ONE_WARPS + 1) * E * sizeof(int);
        const int per = std::max(32, (int)((n + 32 * PL_ONE_WARPS - 1) / (32 * PL_ONE_WARPS)) * 32);
        const auto kernel = plan_place_kernel<PL_ONE_WARPS>;
        if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        return launch_dependent(kernel, 1, 32 * PL_ONE_WARPS, smem, stream, ids, n, per, E, nullptr, nullptr, offs,
                                rows, src);
    }
    const int chunks = (int)plan_chunks(n);
    const size_t smem = (size_t)(PL_CHUNK_WARPS + 1) * E * sizeof(int);
    int32_t* totals = ws + (int64_t)chunks * E;
    cudaError_t e = launch_dependent(plan_count_kernel, chunks, 32 * PL_CHUNK_WARPS, smem, stream, ids, n, E, ws);
    if (e == cudaSuccess)
        e = launch_dependent(plan_scan_kernel, (E + 3) / 4, 128, 0, stream, ws, chunks, E, totals);
    if (e == cudaSuccess)
        e = launch_dependent(plan_place_kernel<PL_CHUNK_WARPS>, chunks, 32 * PL_CHUNK_WARPS, smem, stream, ids, n,
                             PL_CHUNK / PL_CHUNK_WARPS, E, ws, totals, offs, rows, src);
    return e;
}

}  // namespace mxq
