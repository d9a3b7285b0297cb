// The experts' MXFP4 products: y[r] = W[e(r)] . a[row(r)] for rows sorted by
// expert, on the tcgen05 tensor cores (kind::mxf4, block scales of 32 applied
// by the MMA, fp32 accumulation).  E = 1 is a dense product.
//
// One persistent CTA an SM.  A unit is (expert, 128 weight rows, a tile of up
// to nt of the expert's rows); its K runs in stages of 256 columns.  Weights
// are the MMA's 128-row operand and tokens its N operand, so a decode batch
// (one or two rows an expert) wastes no tensor time on padding and the same
// kernel serves one token and a prompt: N is the tile's rows, rounded to 16.
//   warp 0      copies: a stage is a weight tile (16 KiB), a token tile's K
//               block and both scale blocks, all contiguous (bulk copies)
//   warp 1      issues the MMAs (one thread)
//   warps 4..7  epilogue: TMEM -> y, behind the next unit's MMAs (two
//               accumulators)
// Work split: with many units each CTA takes whole ones, round robin.  With
// few, the stages of all units are dealt evenly over the CTAs; a unit cut
// between CTAs leaves fp32 partials in the workspace and the CTA that
// arrives last sums them in the order of K, so the result does not depend on
// which one that is.  No CTA ever waits for another.
#include "moeq_device.cuh"
#include "moeq_mx4_plan.cuh"
#include "moeq_rows.h"

namespace moeq {
namespace {

constexpr int kThreads = kPlanThreads;
constexpr int kMaxStages = 12;
// Whole units from this many a CTA on (below, the stages are dealt evenly).
constexpr int kWholeWaves = 4;
// TMEM columns: accumulators at 0 and 256, the tokens' scales in between and
// the weights' behind.
constexpr int kTmemCols = 512, kAcc1 = 256, kColSfb = 240, kColSfa = 496;

__host__ __device__ constexpr int stage_bytes_of(int nt) {
    return (kMx4TileBytes + nt * 128 + kMx4TileScaleBytes + mx4_tile_scale_bytes(nt) + 1023) / 1024 * 1024;
}

struct Sched {
    int units, kb, grid, cta;
    bool whole;
    long long s0, s1;   // this CTA's stages (dealt mode)
};
struct Part {
    int u, n0, r0, n, kb0, kb1, tile, tiles, e, nb;
};

__device__ __forceinline__ long long deal(long long stages, int c, int grid) { return stages * c / grid; }

// The i-th part of this CTA; false past its last.  A unit's number counts
// experts, then weight blocks, then token tiles: neighbours read the same
// weights.
__device__ __forceinline__ bool part_at(const Sched& s, const Mx4GemmArgs& a, const PlanShared& plan, int i, Part& p) {
    if (s.whole) {
        p.u = s.cta + i * s.grid;
        if (p.u >= s.units) return false;
        p.kb0 = 0;
        p.kb1 = s.kb;
    } else {
        const long long u = s.s0 / s.kb + i;
        const long long lo = u * s.kb > s.s0 ? u * s.kb : s.s0;
        const long long hi = (u + 1) * s.kb < s.s1 ? (u + 1) * s.kb : s.s1;
        if (lo >= hi) return false;
        p.u = static_cast<int>(u);
        p.kb0 = static_cast<int>(lo - u * s.kb);
        p.kb1 = static_cast<int>(hi - u * s.kb);
    }
    const int nbt = mx4_nb(a.N), nt = a.plan.nt;
    const int e = plan_find(plan.tile, a.plan.E, p.u / nbt);  // experts without tiles are never the last such
    const int r0 = plan.first[e], cnt = plan.first[e + 1] - r0;
    const int tiles = plan.tile[e + 1] - plan.tile[e], per = plan_rows_per_tile(cnt, nt);
    const int local = p.u - plan.tile[e] * nbt;
    p.e = e;
    p.tiles = tiles;
    p.nb = local / tiles;
    p.n0 = p.nb * kMx4TileRows;
    const int t = local - p.nb * tiles;
    p.tile = plan.tile[e] + t;
    p.r0 = r0 + t * per;
    p.n = min(per, cnt - t * per);
    return true;
}

// 512 bytes of scales (32 rows of 16 bytes) into four TMEM columns of all four
// lane groups.
__device__ __forceinline__ uint64_t sf_desc(uint32_t smem_addr) {
    uint64_t d = static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(128 >> 4) << 32;  // eight rows of 16 bytes
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// E2M1 operands, E8M0 scales, fp32 accumulator, 128 x N; the scale bytes of
// the MMA's 64 columns are bytes sf and sf + 1 of each row's word.
__device__ __forceinline__ uint32_t idesc_mx4(int n, int sf) {
    return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (1u << 23) | ((128u >> 4) << 24) | (static_cast<uint32_t>(sf) << 29);
}
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        int acc) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
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

// One lane of a converged warp, the same each time.  tcgen05 instructions take
// their operands from uniform registers: under an elected predicate the
// compiler keeps them there, under `lane == 0` it moves them over one by one
// (a stage of 6 scale copies and 4 MMAs of N = 240: 549 cycles against 717).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q; }" : "=r"(p));
    return p != 0;
}
// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return done != 0;
}
// Wait (bounded) for what is in flight after a give-up.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
    const unsigned long long t0 = global_timer_ns();
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

// The sum of a unit's parts for 16 columns, all in the order of K: this CTA's
// own (v) comes from TMEM, the others' from the workspace, two parts' loads
// in flight at a time.  lo_second: the first CTA's part is in its second slot.
__device__ __forceinline__ void sum_parts(const float* __restrict__ part, size_t slot_floats, int c_lo, int c_hi, int own,
                                          int lo_second, int c0, int row, float (&v)[16]) {
    float sum[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) sum[c] = 0.f;
    const size_t at = static_cast<size_t>(c0) * 128 + row * 4;
    for (int k0 = c_lo; k0 <= c_hi; k0 += 2) {
        float4 f[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = k0 + j;
            if (k > c_hi || k == own) continue;
            // only the first of a unit's CTAs can have begun in another unit
            const float* slot = part + (static_cast<size_t>(2 * k) + (k == c_lo ? lo_second : 0)) * slot_floats + at;
#pragma unroll
            for (int c = 0; c < 4; ++c) f[j][c] = __ldcg(reinterpret_cast<const float4*>(slot + c * 512));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = k0 + j;
            if (k > c_hi) continue;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sum[4 * c] += k == own ? v[4 * c] : f[j][c].x;
                sum[4 * c + 1] += k == own ? v[4 * c + 1] : f[j][c].y;
                sum[4 * c + 2] += k == own ? v[4 * c + 2] : f[j][c].z;
                sum[4 * c + 3] += k == own ? v[4 * c + 3] : f[j][c].w;
            }
        }
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] = sum[c];
}

// A step of the epilogue: kCols rows of y (columns of the accumulator) by
// four warps, lane = weight row.  They pass through shared memory, so that a
// row's 128 values leave as 16-byte pieces; where y's rows do not divide so,
// element by element.
template <bool kF32>
struct Epi {
    static constexpr int kCols = kF32 ? 32 : 64;
    static constexpr int kPitch = kF32 ? 528 : 320;  // bytes a row: neighbours in other banks
};
constexpr int kEpiBytes = 64 * 320;
static_assert(Epi<true>::kCols * Epi<true>::kPitch <= kEpiBytes, "one buffer serves both types");

template <bool kF32, int kCols>
__device__ __forceinline__ void store_step(const Mx4GemmArgs& a, const Part& p, int c0, int q, int lane, int n,
                                           const float (&v)[kCols], uint8_t* buf, bool vec) {
    constexpr int kPitch = Epi<kF32>::kPitch;
    if (!vec) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
            if (c0 + c < p.n && n < a.N) store_y<kF32>(a.y, static_cast<int64_t>(p.r0 + c0 + c) * a.ld_y + n, v[c]);
        return;
    }
    named_sync(1, 128);  // the step before has left the buffer
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
    named_sync(1, 128);
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

template <bool kF32>
__global__ void __maxnreg__(160) mx4_gemm_kernel(const __grid_constant__ Mx4GemmArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s, go_s[2], last_s[2];
    __shared__ PlanShared plan;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nt = a.plan.nt;
    const int sfb_bytes = mx4_tile_scale_bytes(nt), sfb_chunk = sfb_bytes / 2;
    const int off_b = kMx4TileBytes, off_sfa = off_b + nt * 128, off_sfb = off_sfa + kMx4TileScaleBytes;
    const int stage_bytes = stage_bytes_of(nt);
    volatile int* abort = &abort_s;

    if (tid == 0) {
        abort_s = 0;
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_s, kTmemCols);
        tc_fence_before();
    }
    plan_scan(a.plan, plan);  // ends in a block barrier
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int nbt = mx4_nb(a.N), total = plan.tile[a.plan.E] * nbt;

    Sched s;
    s.units = total;
    s.kb = mx4_kb(a.K);
    s.cta = blockIdx.x;
    const long long all_stages = static_cast<long long>(total) * s.kb;
    s.grid = static_cast<int>(min(static_cast<long long>(gridDim.x), all_stages));
    s.whole = total >= kWholeWaves * static_cast<int>(gridDim.x);
    s.s0 = s.s1 = 0;
    if (!s.whole && s.cta < s.grid) {
        s.s0 = deal(all_stages, s.cta, s.grid);
        s.s1 = deal(all_stages, s.cta + 1, s.grid);
    }
    auto stage_at = [&](int st) { return smem + st * stage_bytes; };
    auto give_up = [&] {
        *abort = 1;
        if (a.status) atomicExch(a.status, static_cast<int>(MOEQ_ERR_TIMEOUT));
    };

    if (warp == 0) {
        // -------------------------------------------------------- copies
        if (elect_one()) {
            // weights that one token tile reads are not read again; those of
            // several, and the token tiles, come from L2 the next time
            const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
            auto weights = [&](const Part& p, int kb, int st) {
                const int64_t tile = (static_cast<int64_t>(p.e) * nbt + p.nb) * s.kb + kb;
                const uint64_t policy = p.tiles > 1 ? again : once;
                const int n16 = (p.n + 15) & ~15;
                mbar_arrive_expect_tx(&full[st], kMx4TileBytes + kMx4TileScaleBytes + n16 * 128 + sfb_bytes);
                bulk_load(stage_at(st), a.w + tile * kMx4TileBytes, kMx4TileBytes, &full[st], policy);
                bulk_load(stage_at(st) + off_sfa, a.sw + tile * kMx4TileScaleBytes, kMx4TileScaleBytes, &full[st], policy);
            };
            auto tokens = [&](const Part& p, int kb, int st) {
                const int64_t block = static_cast<int64_t>(p.tile) * s.kb + kb;
                const int n16 = (p.n + 15) & ~15;
                bulk_load(stage_at(st) + off_b, a.a + block * nt * 128, n16 * 128, &full[st], again);
                bulk_load(stage_at(st) + off_sfb, a.sa + block * sfb_bytes, sfb_bytes, &full[st], again);
            };
            // The first stages' weights need not wait for the kernel ahead,
            // which writes the token tiles.
            Part p;
            int ahead = 0;
            for (int i = 0; ahead < a.stages && part_at(s, a, plan, i, p); ++i)
                for (int kb = p.kb0; kb < p.kb1 && ahead < a.stages; ++kb) weights(p, kb, ahead++);
            pdl_wait();
            int it = 0, st = 0;
            uint32_t phase = 1;  // of the ring's previous round
            bool ok = true;
            for (int i = 0; ok && part_at(s, a, plan, i, p); ++i)
                for (int kb = p.kb0; kb < p.kb1; ++kb, ++it) {
                    if (it >= ahead) {
                        ok = mbar_wait_bounded(&empty[st], phase, abort);
                        if (!ok) break;
                        weights(p, kb, st);
                    }
                    tokens(p, kb, st);
                    if (++st == a.stages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            if (!ok) {
                give_up();
                // copies in flight land before the CTA may end
                for (int j = max(0, it - a.stages); j < it; ++j) drain(&full[j % a.stages], (j / a.stages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMAs
        // The tensor core's queue holds little: the next stage's barrier is
        // asked for while this one's last MMAs go out.
        if (elect_one()) {
            int st = 0;
            uint32_t phase = 0;
            bool ok = true, ready = false;
            Part p;
            for (int i = 0; ok && part_at(s, a, plan, i, p); ++i) {
                const int buf = i & 1;
                if (i >= 2) ok = mbar_wait_bounded(&acc_empty[buf], ((i >> 1) - 1) & 1, abort);
                const int n16 = (p.n + 15) & ~15;
                const uint32_t d = tmem + buf * kAcc1;
                const uint32_t id0 = idesc_mx4(n16, 0), id2 = idesc_mx4(n16, 2);
                for (int kb = p.kb0; ok && kb < p.kb1; ++kb) {
                    if (!ready) ok = mbar_wait_bounded(&full[st], phase, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sp = smem_u32(stage_at(st));
                    const uint64_t fa = sf_desc(sp + off_sfa), fb = sf_desc(sp + off_sfb);
                    const uint64_t ad = umma_desc_sw128(sp), bd = umma_desc_sw128(sp + off_b);
                    uint64_t* const done = &empty[st];
                    if (++st == a.stages) {
                        st = 0;
                        phase ^= 1;
                    }
#pragma unroll
                    for (int kc = 0; kc < 2; ++kc) {
                        sf_copy(tmem + kColSfa + kc * 4, fa + kc * (512 >> 4));
                        sf_copy(tmem + kColSfb + kc * 8, fb + kc * (sfb_chunk >> 4));
                        if (n16 > 128) sf_copy(tmem + kColSfb + kc * 8 + 4, fb + kc * (sfb_chunk >> 4) + (512 >> 4));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // 64 columns = 32 bytes of a row
                        if (j == 2) ready = mbar_test_wait(&full[st], phase);
                        mma_mx4(d, ad + j * 2, bd + j * 2, j & 1 ? id2 : id0, tmem + kColSfa + (j >> 1) * 4,
                                tmem + kColSfb + (j >> 1) * 8, kb > p.kb0 || j > 0);
                    }
                    umma_commit(done);
                }
                if (ok) umma_commit(&acc_full[buf]);
            }
            if (!ok) {
                give_up();
                umma_commit(&drained);
                drain(&drained, 0);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------- epilogue
        pdl_wait();
        const int q = warp - 4;
        uint8_t* stage_y = smem + a.stages * stage_bytes;
        // rows of y in 16-byte pieces
        const bool vec_y = a.N % (kF32 ? 4 : 8) == 0 && a.ld_y % (kF32 ? 4 : 8) == 0 &&
                           (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
        Part p;
        for (int i = 0; part_at(s, a, plan, i, p); ++i) {
            const int buf = i & 1;
            if (lane == 0 && !mbar_wait_bounded(&acc_full[buf], (i >> 1) & 1, abort)) give_up();
            __syncwarp();
            // One thread decides for all four warps whether to go on: they meet
            // at barriers below.  (Two copies: a slow warp may still read the
            // last unit's.)
            if (tid == 128) {
                go_s[buf] = !*abort;
            }
            named_sync(1, 128);
            if (!go_s[buf]) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * kAcc1 + (static_cast<uint32_t>(q * 32) << 16);
            const int n = p.n0 + q * 32 + lane;
            const size_t slot_floats = static_cast<size_t>(nt) * 128;
            const bool cut = p.kb0 > 0 || p.kb1 < s.kb;
            // the CTAs that hold the unit's stages: c_lo .. c_hi
            int c_lo = s.cta, c_hi = s.cta;
            bool join = false;  // every other part is in the workspace: this CTA sums them
            if (cut) {
                const long long f = static_cast<long long>(p.u) * s.kb, l = f + s.kb - 1;
                while (deal(all_stages, c_lo, s.grid) > f) --c_lo;
                while (deal(all_stages, c_hi + 1, s.grid) <= l) ++c_hi;
                if (tid == 128) last_s[buf] = ld_acquire(a.tickets + p.u) == c_hi - c_lo;
                named_sync(1, 128);
                join = last_s[buf];
                if (!join) {
                    float4* slot = reinterpret_cast<float4*>(
                                       a.part + (static_cast<size_t>(2 * s.cta) + (p.u != s.s0 / s.kb)) * slot_floats) +
                                   q * 32 + lane;
                    for (int c0 = 0; c0 < p.n; c0 += 16) {
                        float v[16];
                        tmem_ld16(acc + c0, v);
                        tmem_wait_ld();
                        tmem_use16(v);
#pragma unroll
                        for (int c = 0; c < 16; c += 4)
                            __stcg(slot + (c0 + c) / 4 * 128, make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]));
                    }
                    __threadfence();
                    named_sync(1, 128);
                    if (tid == 128) last_s[buf] = atom_add_acq_rel(a.tickets + p.u, 1) == c_hi - c_lo;
                    named_sync(1, 128);
                    join = last_s[buf];
                }
                if (join) {
                    __threadfence();
                    if (tid == 128) a.tickets[p.u] = 0;
                }
            }
            auto release = [&] {  // the accumulator is read: the next unit but one may have it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[buf]);
            };
            if (!cut) {
                constexpr int kCols = Epi<kF32>::kCols;
                for (int c0 = 0; c0 < p.n; c0 += kCols) {
                    float v[kCols];  // columns past the tile's are read and not stored
#pragma unroll
                    for (int j = 0; j < kCols; j += 16) tmem_ld16(acc + c0 + j, v + j);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < kCols; j += 16) tmem_use16(v + j);
                    if (c0 + kCols >= p.n) release();
                    store_step<kF32, kCols>(a, p, c0, q, lane, n, v, stage_y, vec_y);
                }
            } else {
                const int lo_second = deal(all_stages, c_lo, s.grid) / s.kb != p.u;
                for (int c0 = 0; join && c0 < p.n; c0 += 16) {
                    float v[16];
                    tmem_ld16(acc + c0, v);
                    tmem_wait_ld();
                    tmem_use16(v);
                    sum_parts(a.part, slot_floats, c_lo, c_hi, s.cta, lo_second, c0, q * 32 + lane, v);
                    store_step<kF32, 16>(a, p, c0, q, lane, n, v, stage_y, vec_y);
                }
                release();
            }
        }
        // rows that belong to no expert
        const int t = tid - 128;
        for (int64_t r = static_cast<int64_t>(plan.first[a.plan.E]) + blockIdx.x; r < a.plan.R; r += gridDim.x)
            for (int c = t; c < a.N; c += 128) store_y<kF32>(a.y, r * a.ld_y + c, 0.f);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

// Rows of a token tile.  About twice the average of an expert, so that most
// experts are one tile (its weights then stream once), but no wider than
// that: a narrow tile leaves shared memory to more weight stages in flight.
int mx4_tile_rows(int R, int E) {
    const long long want = 2LL * R / E + 16;
    const int r16 = (R + 15) / 16 * 16;
    const int w16 = static_cast<int>(want > kMx4MaxTileRows ? kMx4MaxTileRows : (want + 15) / 16 * 16);
    const int nt = E == 1 ? r16 : w16;
    return nt < r16 ? (nt > kMx4MaxTileRows ? kMx4MaxTileRows : nt) : (r16 > kMx4MaxTileRows ? kMx4MaxTileRows : r16);
}

cudaError_t launch_mx4_gemm(Mx4GemmArgs a, int grid, bool pdl, cudaStream_t stream) {
    const int sb = stage_bytes_of(a.plan.nt);
    // of 227 KiB: less the static arrays, the alignment and the epilogue's buffers
    const int budget = 216 * 1024 - kEpiBytes;
    a.stages = budget / sb < kMaxStages ? budget / sb : kMaxStages;
    const int smem = a.stages * sb + kEpiBytes + 1024;
    auto kern = a.y_f32 ? mx4_gemm_kernel<true> : mx4_gemm_kernel<false>;
    static SmemOnce once[2];
    const cudaError_t e = once[a.y_f32 != 0].raise(reinterpret_cast<const void*>(kern), budget + kEpiBytes + 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace moeq
