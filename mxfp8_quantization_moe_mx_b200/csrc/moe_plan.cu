// moe_plan.cu -- from the experts of each token to the rows of the grouped products
// (sm_100a).
//
// ids (n = T * k values in 0..E-1, or out of range: routed nowhere) -> a stable sort by
// expert: row r of the grouped operand holds slot src[r] (token src[r] / k), group e is
// rows [offs[e-1], offs[e]), rows[slot] is the slot's row or -1.  A counting sort:
//   one CTA (n <= PL_ONE) keeps everything in shared memory: every warp counts its run of
//   consecutive slots by expert, the counts become starts, every slot takes its row.
//   Else CTAs take consecutive chunks of slots in two launches, the second dependent on the
//   first: count writes the chunks' counts to the workspace, [E][chunks]; place reads them
//   all (at most 148 chunks, a warp per expert), adds up those of the
//   earlier chunks and of all, and goes on as the one CTA does.
// Counting is by shared-memory atomics, whose order does not show.  Ranks among 32
// neighbouring slots come from a word per expert in which each lane sets its bit, so the
// rows are in the order of the slots and no atomic decides them (a match of equal ids
// instead, __match_any_sync, cost 30 us for 22: its time grows with the distinct values).
//
// The bytes (12 per slot) are few: what it costs is the launches and the latency of each
// step, and for many slots the counts, which every CTA of place reads whole before it can place
// any (524288 slots, 256 experts: 150 KB a CTA, 22 MB of the 26 that come from L2; 15 us).

#include <algorithm>

#include "dependent.cuh"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int PL_WARPS = 16;
constexpr int PL_ONE = 8192;        // slots that one CTA takes, at most 512 per warp
constexpr int PL_MIN_PER = 128;     // more: at least 128 slots per warp, ...
constexpr int PL_MAX_CHUNKS = 148;  // ... in at most one CTA per SM

constexpr int PL_BATCH = 8;  // steps of 32 slots whose ids are loaded together

// The experts of the lane's slots first + lane, + 32, ... below end; -1 where there is none.
__device__ __forceinline__ void load_batch(const int32_t* __restrict__ ids, int64_t first, int64_t end, int E,
                                           int lane, int (&id)[PL_BATCH]) {
#pragma unroll
    for (int i = 0; i < PL_BATCH; ++i) {
        const int64_t at = first + 32 * i + lane;
        id[i] = at < end ? __ldg(ids + at) : -1;
    }
#pragma unroll
    for (int i = 0; i < PL_BATCH; ++i)
        if (id[i] >= E) id[i] = -1;
}

// The warp's slots [first, end) by expert, added to cnt[0..E) (shared).
__device__ __forceinline__ void count_slots(const int32_t* __restrict__ ids, int64_t first, int64_t end, int E,
                                            int* cnt, int lane) {
    for (int64_t a = first; a < end; a += 32 * PL_BATCH) {
        int id[PL_BATCH];
        load_batch(ids, a, end, E, lane, id);
#pragma unroll
        for (int i = 0; i < PL_BATCH; ++i)
            if (id[i] >= 0) atomicAdd(cnt + id[i], 1);
    }
}

__global__ void __launch_bounds__(32 * PL_WARPS) plan_count_kernel(const int32_t* __restrict__ ids, int64_t n, int per,
                                                                   int E, int32_t* __restrict__ counts) {
    extern __shared__ int plan_s[];
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < E; e += 32 * PL_WARPS) plan_s[e] = 0;
    __syncthreads();
    const int64_t first = ((int64_t)blockIdx.x * PL_WARPS + warp) * per;
    count_slots(ids, first, min(n, first + per), E, plan_s, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 32 * PL_WARPS) counts[(int64_t)e * gridDim.x + blockIdx.x] = plan_s[e];
}

__device__ __forceinline__ int redux_add(int v) { return __reduce_add_sync(FULL_MASK, v); }

// A warp takes `per` consecutive slots.  counts: NULL for the one CTA that has all slots.
__global__ void __launch_bounds__(32 * PL_WARPS) plan_place_kernel(const int32_t* __restrict__ ids, int64_t n, int per,
                                                                int E, const int32_t* __restrict__ counts,
                                                                int32_t* __restrict__ offs, int32_t* __restrict__ rows,
                                                                int32_t* __restrict__ src) {
    extern __shared__ int plan_s[];  // [PL_WARPS][E] counts, then starts; [E] totals, then expert starts; [E] earlier;
                                // [PL_WARPS][E] lanes of an expert
    __shared__ int routed_s;
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* starts = plan_s + PL_WARPS * E;
    int* before = starts + E;
    int* mine = plan_s + warp * E;
    unsigned* mask = reinterpret_cast<unsigned*>(before + E) + warp * E;
    const int64_t first = ((int64_t)blockIdx.x * PL_WARPS + warp) * per, end = min(n, first + per);
    for (int e = lane; e < E; e += 32) mine[e] = 0, mask[e] = 0;
    __syncwarp();
    count_slots(ids, first, end, E, mine, lane);
    if (counts) {
        const int chunks = gridDim.x;
        constexpr int L = (PL_MAX_CHUNKS + 31) / 32, B = 4;  // B experts' counts in flight
        for (int e0 = warp; e0 < E; e0 += B * PL_WARPS) {
            int v[B][L];
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int j = 0; j < L; ++j) {
                    const int e = e0 + i * PL_WARPS, c = 32 * j + lane;
                    v[i][j] = e < E && c < chunks ? __ldg(counts + (int64_t)e * chunks + c) : 0;
                }
#pragma unroll
            for (int i = 0; i < B; ++i) {
                int all = 0, early = 0;
#pragma unroll
                for (int j = 0; j < L; ++j) {
                    all += v[i][j];
                    early += 32 * j + lane < (int)blockIdx.x ? v[i][j] : 0;
                }
                all = redux_add(all);
                early = redux_add(early);
                const int e = e0 + i * PL_WARPS;
                if (lane == 0 && e < E) {
                    starts[e] = all;
                    before[e] = early;
                }
            }
        }
    }
    __syncthreads();
    // per expert: the warps' counts become starts relative to the expert's
    for (int e = threadIdx.x; e < E; e += 32 * PL_WARPS) {
        int run = counts ? before[e] : 0;
#pragma unroll
        for (int w = 0; w < PL_WARPS; ++w) {
            const int v = plan_s[w * E + e];
            plan_s[w * E + e] = run;
            run += v;
        }
        if (!counts) starts[e] = run;
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
    for (int64_t a = first; a < end; a += 32 * PL_BATCH) {
        int ids_[PL_BATCH];
        load_batch(ids, a, end, E, lane, ids_);
#pragma unroll
        for (int i = 0; i < PL_BATCH; ++i) {
            const int64_t at = a + 32 * i + lane;
            const int id = ids_[i];
            if (id >= 0) atomicOr(mask + id, 1u << lane);
            __syncwarp();
            int r = -1, base = 0;
            unsigned same = 0;
            if (id >= 0) {
                same = mask[id];
                base = mine[id];
                r = starts[id] + base + __popc(same & ((1u << lane) - 1u));
            }
            __syncwarp();
            if (id >= 0 && lane == __ffs(same) - 1) {
                mask[id] = 0;
                mine[id] = base + __popc(same);
            }
            __syncwarp();
            if (at < end) {
                rows[at] = r;
                if (r >= 0) src[r] = (int32_t)at;
                if (at >= routed) src[at] = -1;  // rows behind the last group
            }
        }
    }
}

// Slots per warp and chunks of n > PL_ONE slots.
struct PlanShape {
    int per, chunks;
};
PlanShape plan_shape(int64_t n) {
    const int64_t warps = (int64_t)PL_MAX_CHUNKS * PL_WARPS;
    const int64_t per = std::max<int64_t>(PL_MIN_PER, ((n + warps - 1) / warps + 31) / 32 * 32);
    return {(int)per, (int)((n + per * PL_WARPS - 1) / (per * PL_WARPS))};
}

}  // namespace

// The one CTA needs none: its counts never leave it.
int64_t plan_workspace_bytes(int64_t n, int E) { return n <= PL_ONE ? 0 : 4 * (int64_t)plan_shape(n).chunks * E; }

cudaError_t launch_moe_plan(const int32_t* ids, int64_t n, int E, int32_t* offs, int32_t* rows, int32_t* src,
                            int32_t* ws, cudaStream_t stream) {
    constexpr int PER_EXPERT = (2 * PL_WARPS + 2) * (int)sizeof(int), MAX_SMEM = 1024 * PER_EXPERT;  // 136 KB
    const size_t smem = (size_t)E * PER_EXPERT;
    // Without this opt-in the static memory counts within the 48 KB, too.  It stays with the
    // kernel, and other host threads launch it: always the same value, never a call's own.
    if (smem > 47 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(plan_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
        if (e != cudaSuccess) return e;
    }
    if (n <= PL_ONE) {
        const int per = std::max(32, (int)((n + 32 * PL_WARPS - 1) / (32 * PL_WARPS)) * 32);
        return launch_dependent(plan_place_kernel, 1, 32 * PL_WARPS, smem, stream, ids, n, per, E, nullptr, offs, rows,
                                src);
    }
    const PlanShape sh = plan_shape(n);
    const cudaError_t e = launch_dependent(plan_count_kernel, sh.chunks, 32 * PL_WARPS, (size_t)E * sizeof(int),
                                           stream, ids, n, sh.per, E, ws);
    if (e != cudaSuccess) return e;
    return launch_dependent(plan_place_kernel, sh.chunks, 32 * PL_WARPS, smem, stream, ids, n, sh.per, E,
                            ws, offs, rows, src);
}

}  // namespace mxq
