// The token tiles of a grouped product, from the experts' row ranges: shared
// by the kernel that fills the tiles and the one that multiplies them.
#pragma once

#include "moeq_device.cuh"
#include "moeq_rows.h"

namespace moeq {

constexpr int kPlanThreads = 256;  // four experts a thread: MOEQ_MAX_EXPERTS

// In shared memory: plan_ints(E) ints.
struct PlanShared {
    int* first;  // [E + 1] first row of each expert, clamped to [0, R] and made to rise
    int* tile;   // [E + 1] token tiles before each expert
    int* warp;   // [2][kPlanThreads / 32]
};
__host__ __device__ constexpr int plan_ints(int E) { return 2 * (E + 1) + 2 * (kPlanThreads / 32); }
__device__ __forceinline__ PlanShared plan_at(int* mem, int E) {
    return {mem, mem + E + 1, mem + 2 * (E + 1)};
}

// Rows are given to experts by `offs`; values out of range or order are
// clamped, so that no row, tile or buffer index leaves its range.  Called by
// all threads of a block of at least kPlanThreads.  `offs` is read from L2,
// where its writer left it: the product scans the plan ahead of its own
// griddepcontrol.wait (the kernel between it and that writer let it start only
// once that writer had ended).
__device__ __forceinline__ void plan_scan(const Mx4Plan& p, const PlanShared& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool mine_too = tid < kPlanThreads;
    int top[4], run = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = tid * 4 + i;
        if (e <= p.E) run = max(run, min(max(__ldcg(p.offs + e), 0), p.R));
        top[i] = run;
    }
    int inc = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) inc = max(inc, __shfl_up_sync(0xffffffffu, inc, o));
    if (lane == 31 && mine_too) s.warp[warp] = inc;
    int before = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    for (int w = 0; w < warp && mine_too; ++w) before = max(before, s.warp[w]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (mine_too && tid * 4 + i <= p.E) s.first[tid * 4 + i] = max(before, top[i]);
    if (tid == kPlanThreads - 1 && p.E == MOEQ_MAX_EXPERTS)
        s.first[p.E] = max(max(before, run), min(max(__ldcg(p.offs + p.E), 0), p.R));
    __syncthreads();
    int sum = 0, mine[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = tid * 4 + i;
        mine[i] = sum;
        if (mine_too && e < p.E) sum += (s.first[e + 1] - s.first[e] + p.nt - 1) / p.nt;
    }
    inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31 && mine_too) s.warp[kPlanThreads / 32 + warp] = inc;
    __syncthreads();
    before = inc - sum;
    for (int w = 0; w < warp && mine_too; ++w) before += s.warp[kPlanThreads / 32 + w];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (mine_too && tid * 4 + i < p.E) s.tile[tid * 4 + i] = before + mine[i];
    if (tid == kPlanThreads - 1) s.tile[p.E] = before + sum;
    __syncthreads();
}

// The last index e of v[0 .. n - 1] (rising) with v[e] <= x; v[0] <= x.
__device__ __forceinline__ int plan_find(const int* v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// An expert's rows are shared out evenly over its tiles, `align` (16 or 32) at
// a time.
__device__ __forceinline__ int plan_rows_per_tile(int rows, int nt, int align) {
    const int tiles = max((rows + nt - 1) / nt, 1);
    return ((rows + tiles - 1) / tiles + align - 1) & ~(align - 1);
}

}  // namespace moeq
