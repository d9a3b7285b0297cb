// Building blocks of the products that run on one CTA or on a pair of them
// (a cluster whose two SMs share a tcgen05 tile): barriers and commits across
// the pair, TMEM, the epilogue that turns an accumulator's columns into rows,
// and the driver's tensor-map encoder.
#pragma once

#include <cuda.h>

#include "moeq_device.cuh"

namespace moeq {

constexpr int kTmemCols = 512;

// Four warps for copies and MMAs, and four of epilogue for each group: a
// pair's short MXFP4 units (eight stages at K = 2048) end faster than one
// group stores them, so there two groups take turns.
__host__ __device__ constexpr int epi_groups(bool pair) { return pair ? 2 : 1; }
__host__ __device__ constexpr int threads_of(bool pair) { return 128 + 128 * epi_groups(pair); }

// One arrival on `bar` (in both CTAs of a pair) when everything issued so far
// has completed.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    if constexpr (kPair)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        umma_commit(bar);
}
template <bool kPair>
__device__ __forceinline__ void tmem_take(uint32_t* smem_dst) {
    if constexpr (kPair) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(smem_dst, kTmemCols);
    }
}
template <bool kPair>
__device__ __forceinline__ void tmem_give(uint32_t taddr) {
    if constexpr (kPair)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kTmemCols) : "memory");
    else
        tmem_dealloc(taddr, kTmemCols);
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// This barrier's address in the first CTA of the pair.
__device__ __forceinline__ uint32_t in_first(uint64_t* bar) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
    return r;
}
// An arrival on the first CTA's barrier at this offset.
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
    asm volatile(
        "{ .reg .b32 r; mapa.shared::cluster.u32 r, %0, 0;\nmbarrier.arrive.release.cluster.shared::cluster.b64 _, [r]; }" ::"r"(
            smem_u32(bar))
        : "memory");
}
// As mbar_wait_bounded, seeing what the other CTA of the pair released.
__device__ __forceinline__ bool cluster_try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool cluster_wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (cluster_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (cluster_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0 && (*abort || global_timer_ns() - t0 > kWaitLimitNs)) return false;
    }
}

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}
// 16 accumulator columns of this thread's lane, valid after tmem_wait_ld and
// (so that no use moves above the wait) tmem_use16.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_use16(float* v) {
    asm volatile(""
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One lane of a converged warp, the same each time.  Issued under it, a stage
// of 6 scale copies and 4 MMAs takes 510 cycles at N = 208 by one CTA and 449
// at N = 224 by a pair; under `lane == 0` both take 718.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q; }" : "=r"(p));
    return p != 0;
}
// Whether a phase is complete, without waiting.
template <bool kPair>
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    if constexpr (kPair)
        asm volatile(
            "{ .reg .pred p; mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    else
        asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(done)
                     : "r"(smem_u32(bar)), "r"(parity)
                     : "memory");
    return done != 0;
}
// Wait (bounded, from t0 on) for what is in flight after a give-up.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, unsigned long long t0) {
    while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kWaitLimitNs) {
    }
}

template <bool kF32>
__device__ __forceinline__ void store_y(void* y, int64_t at, float v) {
    if constexpr (kF32)
        static_cast<float*>(y)[at] = v;
    else
        static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
}

// A step of the epilogue: kCols rows of y (columns of the accumulator) by
// four warps, lane = weight row.  They pass through shared memory, so that a
// row's 128 values leave as 16-byte pieces; where y's rows do not divide so,
// element by element.
template <bool kF32>
struct Epi {
    static constexpr int kPitch = kF32 ? 528 : 320;  // bytes a row: neighbours in other banks
};
// Columns a step.  A pair takes half as many: its two groups' buffers then
// leave room for a sixth stage of the widest tiles.
__host__ __device__ constexpr int epi_cols(bool f32, bool pair) { return (f32 ? 32 : 64) / (pair ? 2 : 1); }
__host__ __device__ constexpr int epi_bytes(bool pair) { return epi_cols(false, pair) * Epi<false>::kPitch; }
static_assert(epi_cols(true, false) * Epi<true>::kPitch <= epi_bytes(false) &&
                  epi_cols(true, true) * Epi<true>::kPitch <= epi_bytes(true) && epi_bytes(true) % 16 == 0,
              "one buffer serves both types");

template <bool kF32, int kCols, typename Args, typename Part>
__device__ __forceinline__ void store_step(const Args& a, const Part& p, int c0, int q, int lane, int n,
                                           const float (&v)[kCols], uint8_t* buf, bool vec, int bar) {
    constexpr int kPitch = Epi<kF32>::kPitch;
    if (!vec) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
            if (c0 + c < p.n && n < a.N) store_y<kF32>(a.y, static_cast<int64_t>(p.r0 + c0 + c) * a.ld_y + n, v[c]);
        return;
    }
    named_sync(bar, 128);  // the step before has left the buffer
    if constexpr (kF32) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) *reinterpret_cast<float*>(buf + c * kPitch + (q * 32 + lane) * 4) = v[c];
    } else {
        // a lane pair swaps halves: the even one keeps row c, the odd c + 1
        const bool odd = lane & 1;
        uint8_t* at = buf + odd * kPitch + (q * 32 + (lane & ~1)) * 2;
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[c] : v[c + 1], 1);
            *reinterpret_cast<__nv_bfloat162*>(at + c * kPitch) =
                odd ? __floats2bfloat162_rn(got, v[c + 1]) : __floats2bfloat162_rn(v[c], got);
        }
    }
    named_sync(bar, 128);
    constexpr int kPer = kF32 ? 4 : 8, kPieces = 128 / kPer, kRows = 128 / kPieces;  // of a piece; of a row; at a time
    const int t = q * 32 + lane, piece = t % kPieces, c1 = t / kPieces;
    if (p.n0 + piece * kPer >= a.N) return;
    uint8_t* y = static_cast<uint8_t*>(a.y) +
                 (static_cast<int64_t>(p.r0 + c0 + c1) * a.ld_y + p.n0 + piece * kPer) * (kF32 ? 4 : 2);
    const int64_t step = a.ld_y * (kRows * (kF32 ? 4 : 2));
    uint4 w[kCols / kRows];
#pragma unroll
    for (int i = 0; i < kCols / kRows; ++i) w[i] = *reinterpret_cast<const uint4*>(buf + (c1 + i * kRows) * kPitch + piece * 16);
#pragma unroll
    for (int i = 0; i < kCols / kRows; ++i)
        if (c0 + c1 + i * kRows < p.n) *reinterpret_cast<uint4*>(y + i * step) = w[i];
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (the library links the runtime only).
inline EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

}  // namespace moeq
