// moe_plan.cu -- from the experts of each token to the rows of the grouped products
// (sm_100a).
//
// ids (n = T * k values in 0..E-1, or out of range: routed nowhere) -> a stable sort by
// expert: row r of the grouped operand holds slot src[r] (token src[r] / k), group e is
// rows [offs[e-1], offs[e]), rows[slot] is the slot's row or -1.  Counting sort in two
// passes over the ids:
//   count   a CTA per chunk of PL_CHUNK slots: the chunk's count of every expert, to the
//           workspace, [chunk][E];
//   scan    (more than one chunk) one warp per 32 experts walks the chunks and replaces
//           counts by the number of slots of that expert in earlier chunks; the totals
//           follow in the workspace;
//   place   a CTA per chunk: expert starts from the totals, then every slot's row = start +
//           earlier chunks' + earlier warps' + rank within the warp.
// A warp owns PL_CHUNK / 8 consecutive slots, and ranks among 32 neighbouring slots come
// from a match of equal ids, so the order is that of the slots and no atomic decides it.

#include <algorithm>

#include "mxq_device.cuh"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int PL_WARPS = 8;
constexpr int PL_CHUNK = 2048;
constexpr int PL_STEPS = PL_CHUNK / (32 * PL_WARPS);

// Counts of the warp's slots by expert into cnt[0..E) (shared, zeroed by the warp).
__device__ __forceinline__ void warp_count(const int (&id)[PL_STEPS], int E, int* cnt, int lane) {
    for (int e = lane; e < E; e += 32) cnt[e] = 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PL_STEPS; ++i) {
        const unsigned same = __match_any_sync(FULL_MASK, id[i]);
        if (id[i] >= 0 && lane == __ffs(same) - 1) cnt[id[i]] += __popc(same);
        __syncwarp();
    }
}

__device__ __forceinline__ void load_ids(const int32_t* __restrict__ ids, int64_t n, int E, int64_t first, int lane,
                                         int (&id)[PL_STEPS]) {
#pragma unroll
    for (int i = 0; i < PL_STEPS; ++i) {
        const int64_t at = first + 32 * i + lane;
        int v = at < n ? __ldg(ids + at) : -1;
        if (v < 0 || v >= E) v = -1;
        id[i] = v;
    }
}

__global__ void __launch_bounds__(32 * PL_WARPS) plan_count_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                   int32_t* __restrict__ counts) {
    extern __shared__ int plan_s[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int id[PL_STEPS];
    load_ids(ids, n, E, (int64_t)blockIdx.x * PL_CHUNK + warp * (PL_CHUNK / PL_WARPS), lane, id);
    warp_count(id, E, plan_s + warp * E, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 32 * PL_WARPS) {
        int c = 0;
#pragma unroll
        for (int w = 0; w < PL_WARPS; ++w) c += plan_s[w * E + e];
        counts[(int64_t)blockIdx.x * E + e] = c;
    }
}

// counts[chunk][e] -> slots of e in earlier chunks; counts[chunks][e] = total.
__global__ void __launch_bounds__(32) plan_scan_kernel(int32_t* __restrict__ counts, int chunks, int E) {
    const int e = blockIdx.x * 32 + threadIdx.x;
    if (e >= E) return;
    int run = 0;
    for (int c = 0; c < chunks; ++c) {
        const int v = counts[(int64_t)c * E + e];
        counts[(int64_t)c * E + e] = run;
        run += v;
    }
    counts[(int64_t)chunks * E + e] = run;
}

// `before` / `totals`: NULL when there is one chunk (both come from its own counts).
__global__ void __launch_bounds__(32 * PL_WARPS) plan_place_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                   const int32_t* __restrict__ before,
                                                                   const int32_t* __restrict__ totals,
                                                                   int32_t* __restrict__ offs,
                                                                   int32_t* __restrict__ rows,
                                                                   int32_t* __restrict__ src) {
    extern __shared__ int plan_s[];  // [PL_WARPS][E] counts, then starts; [E] expert starts
    __shared__ int routed_s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* starts = plan_s + PL_WARPS * E;
    const int64_t first = (int64_t)blockIdx.x * PL_CHUNK + warp * (PL_CHUNK / PL_WARPS);
    int id[PL_STEPS];
    load_ids(ids, n, E, first, lane, id);
    warp_count(id, E, plan_s + warp * E, lane);
    __syncthreads();
    // per expert: turn the warps' counts into starts relative to the chunk, keep its total
    for (int e = threadIdx.x; e < E; e += 32 * PL_WARPS) {
        int run = before ? before[(int64_t)blockIdx.x * E + e] : 0;
#pragma unroll
        for (int w = 0; w < PL_WARPS; ++w) {
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
    int* mine = plan_s + warp * E;
#pragma unroll
    for (int i = 0; i < PL_STEPS; ++i) {
        const unsigned same = __match_any_sync(FULL_MASK, id[i]);
        const int64_t at = first + 32 * i + lane;
        int r = -1;
        if (id[i] >= 0) r = starts[id[i]] + mine[id[i]] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (id[i] >= 0 && lane == __ffs(same) - 1) mine[id[i]] += __popc(same);
        __syncwarp();
        if (at < n) {
            rows[at] = r;
            if (r >= 0) src[r] = (int32_t)at;
            if (at >= routed_s) src[at] = -1;  // rows behind the last group
        }
    }
}

}  // namespace

// One chunk needs none: its counts never leave the CTA.
int64_t plan_workspace_bytes(int64_t n, int E) {
    const int64_t chunks = (n + PL_CHUNK - 1) / PL_CHUNK;
    return chunks <= 1 ? 0 : 4 * (chunks + 1) * E;
}

cudaError_t launch_moe_plan(const int32_t* ids, int64_t n, int E, int32_t* offs, int32_t* rows, int32_t* src,
                            int32_t* ws, cudaStream_t stream) {
    const int64_t chunks = std::max<int64_t>(1, (n + PL_CHUNK - 1) / PL_CHUNK);
    const size_t smem = (size_t)(PL_WARPS + 1) * E * sizeof(int);
    const int threads = 32 * PL_WARPS;
    if (chunks == 1) {
        plan_place_kernel<<<1, threads, smem, stream>>>(ids, n, E, nullptr, nullptr, offs, rows, src);
        return cudaGetLastError();
    }
    plan_count_kernel<<<(unsigned)chunks, threads, smem, stream>>>(ids, n, E, ws);
    plan_scan_kernel<<<(unsigned)((E + 31) / 32), 32, 0, stream>>>(ws, (int)chunks, E);
    plan_place_kernel<<<(unsigned)chunks, threads, smem, stream>>>(ids, n, E, ws, ws + chunks * E, offs, rows, src);
    return cudaGetLastError();
}

}  // namespace mxq
