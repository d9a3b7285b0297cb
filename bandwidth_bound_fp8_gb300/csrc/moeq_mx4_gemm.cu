// The experts' MXFP4 products: y[r] = W[e(r)] . a[row(r)] for rows sorted by
// expert, on the tcgen05 tensor cores (kind::mxf4, block scales of 32 applied
// by the MMA, fp32 accumulation).  E = 1 is a dense product.
//
// One persistent CTA an SM.  A unit is (expert, 128 weight rows, a tile of up
// to nt of the expert's rows); its K runs in stages of 256 columns.  Weights
// are the MMA's 128-row operand and tokens its N operand, so a decode batch
// (one or two rows an expert) wastes no tensor time on padding and the same
// kernel serves one token and a prompt: N is the tile's rows, rounded to 16.
//   warps 0, 2  copies: a stage is a weight tile (16 KiB), a token tile's K
//               block and both scale blocks, all contiguous
//   warp 1      issues the MMAs (one thread); warp 3 tells it the parts
//   warps 4..7  epilogue: TMEM -> y, behind the next unit's MMAs (two
//               accumulators)
// Work split: each CTA (or pair) takes whole units, round robin.  A few units
// of long K are cut in four along K: the parts leave fp32 sums in the
// workspace and the CTA that arrives last adds them in the order of K, so the
// result does not depend on which one that is.  No CTA ever waits for another.
#include "moeq_device.cuh"
#include "moeq_mx4_plan.cuh"
#include "moeq_pair.cuh"
#include "moeq_rows.h"

namespace moeq {
namespace {

static_assert(threads_of(false) >= kPlanThreads, "the plan's scan needs its threads");
// Stages in flight at most.  Seven of a narrow tile's (17 KiB of weights each)
// keep HBM busy; with more, its throughput falls again: 61 tokens over 256
// experts take 294 us with 6, 300 with 7, 313 with 9; one token 22.9, 22.4 and
// 22.1; an LM head of 6144 x 151552 72.5, 72.5 and 75.1.
constexpr int kMaxStages = 7;
// Tiles of this many rows or more are multiplied by pairs of CTAs; their most
// rows (a multiple of 32).  8192 tokens over 256 experts (K 6144, N 4096):
// 867 us in pairs, 953 without; 64 experts of about 50 to 200 rows (K 2048,
// N 2816): equal within 2 %.
constexpr int kPairRows = 200, kPairTileRows = 224;
// Most rows of one CTA's tile.
constexpr int kSingleTileRows = (kPairRows + 14) / 16 * 16;
// Units are cut in kCut parts where that many of them have a worker each and K
// is long enough for the join to pay: a part saves about 0.2 us for every K
// block, the join costs 2 us and 1.6 us for every 16 rows of the tile.
// 1 x 32768 -> 128: 36 us whole; 160 x 6144 -> 1024: 15 us whole, 62 with the
// stages dealt to all SMs; one token over eight experts (256 units): 22.4 us
// whole, 28 with the stages dealt evenly, although half the SMs take one
// unit and half two (the others' bandwidth goes to them).
constexpr int kCut = 4;
__host__ __device__ constexpr bool cut_pays(int units, int kb, int nt, int workers) {
    return units * kCut <= workers && kb >= 8 + nt / 2;
}
// TMEM columns: accumulators at 0 and 256, the tokens' scales in between and
// the weights' behind.
constexpr int kAcc1 = 256, kColSfb = 240, kColSfa = 496;
static_assert(kSingleTileRows == 208 && kSingleTileRows <= kColSfb && kPairTileRows <= kColSfb &&
                  kAcc1 + kPairTileRows <= kColSfa && kAcc1 + kSingleTileRows <= kColSfa,
              "accumulators end before the scales");

__host__ __device__ constexpr int stage_bytes_of(int nt, bool pair) {
    return (kMx4TileBytes + nt / (pair ? 2 : 1) * 128 + kMx4TileScaleBytes + mx4_tile_scale_bytes(nt) + 1023) / 1024 * 1024;
}

struct Sched {
    int units, kb, grid, cta;  // cta, grid: of pairs where two CTAs share a unit
    int nbu, rank;             // weight units of a tile (blocks of 128 rows, or pairs of them); this CTA of its pair
    bool cut;
};
struct Part {
    int u, n0, r0, n, n_mma, kb0, kb1, tile, tiles, e, nb;
};

// The i-th part of this CTA; false past its last.  A unit's number counts
// experts, then weight blocks, then token tiles: neighbours read the same
// weights.
__device__ __forceinline__ bool part_at(const Sched& s, const Mx4GemmArgs& a, const PlanShared& plan, int i, Part& p) {
    p.u = s.cut ? s.cta / kCut : s.cta + i * s.grid;
    if (p.u >= s.units || (s.cut && i > 0)) return false;
    const int c = s.cta % kCut;
    p.kb0 = s.cut ? s.kb * c / kCut : 0;
    p.kb1 = s.cut ? s.kb * (c + 1) / kCut : s.kb;
    const int nt = a.plan.nt, align = a.plan.align;
    const int e = plan_find(plan.tile, a.plan.E, p.u / s.nbu);  // experts without tiles are never the last such
    const int r0 = plan.first[e], cnt = plan.first[e + 1] - r0;
    const int tiles = plan.tile[e + 1] - plan.tile[e], per = plan_rows_per_tile(cnt, nt, align);
    const int local = p.u - plan.tile[e] * s.nbu, nbu = local / tiles, t = local - nbu * tiles;
    p.e = e;
    p.tiles = tiles;
    p.nb = align == 32 ? 2 * nbu + s.rank : nbu;
    p.n0 = p.nb * kMx4TileRows;
    p.tile = plan.tile[e] + t;
    p.r0 = r0 + t * per;
    p.n = min(per, cnt - t * per);
    p.n_mma = (p.n + align - 1) & ~(align - 1);
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
// With kPair the instructions act on a pair of CTAs (one cluster): issued by
// the first, they read shared memory and write TMEM at the same offsets in
// both.
template <bool kPair>
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint64_t desc) {
    if constexpr (kPair)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// E2M1 operands, E8M0 scales, fp32 accumulator, m x n; the scale bytes of the
// MMA's 64 columns are bytes sf and sf + 1 of each row's word.
__device__ __forceinline__ uint32_t idesc_mx4(int m, int n, int sf) {
    return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24) | (static_cast<uint32_t>(sf) << 29);
}
template <bool kPair>
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        int acc) {
    if constexpr (kPair)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
            : "memory");
}
// Rows y .. of a matrix of 128-byte rows into this CTA's shared memory,
// counted on a barrier of either CTA of the pair (which only tensor copies
// can do; a thread that passed the news on took 1200 cycles a stage for its
// release).
__device__ __forceinline__ void rows_load(void* dst, const CUtensorMap* map, int y, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar), "l"(policy)
        : "memory");
}
// The sum of a unit's parts for 16 columns, in the order of K: this CTA's own
// (v) comes from TMEM, the others' from the workspace, two parts' loads in
// flight at a time.  part: the unit's first part, this thread's row.
__device__ __forceinline__ void sum_parts(const float* __restrict__ part, size_t part_floats, int own, int c0,
                                          float (&v)[16]) {
    float sum[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) sum[c] = 0.f;
#pragma unroll
    for (int k0 = 0; k0 < kCut; k0 += 2) {
        float4 f[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (k0 + j != own) {
                const float* at = part + (k0 + j) * part_floats + static_cast<size_t>(c0) * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c) f[j][c] = __ldcg(reinterpret_cast<const float4*>(at + c * 512));
            }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bool mine = k0 + j == own;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sum[4 * c] += mine ? v[4 * c] : f[j][c].x;
                sum[4 * c + 1] += mine ? v[4 * c + 1] : f[j][c].y;
                sum[4 * c + 2] += mine ? v[4 * c + 2] : f[j][c].z;
                sum[4 * c + 3] += mine ? v[4 * c + 3] : f[j][c].w;
            }
        }
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] = sum[c];
}

// The operands as matrices of 128-byte rows, for a pair's copies: the box is
// what one copy takes.
struct PairMaps {
    CUtensorMap w, sw, sa;                 // 128 rows, 8, and a K block's token scales
    CUtensorMap a[kPairTileRows / 2 / 16];  // 16 rows, 32, ...
};
struct NoMaps {};
template <bool kPair>
struct MapsOf {
    using type = NoMaps;
};
template <>
struct MapsOf<true> {
    using type = PairMaps;
};

template <bool kF32, bool kPair>
__global__ void __maxnreg__(160)
    mx4_gemm_kernel(const __grid_constant__ Mx4GemmArgs a, const __grid_constant__ typename MapsOf<kPair>::type maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint64_t part_full[4], part_empty[4];
    __shared__ int part_ring[4];
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s, go_s[2][2], last_s[2][2];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nt = a.plan.nt;
    const int sfb_bytes = mx4_tile_scale_bytes(nt), sfb_chunk = sfb_bytes / 2;
    const int off_b = kMx4TileBytes, off_sfa = off_b + nt / (kPair ? 2 : 1) * 128, off_sfb = off_sfa + kMx4TileScaleBytes;
    const int stage_bytes = stage_bytes_of(nt, kPair);
    const int rank = kPair ? static_cast<int>(cluster_rank()) : 0;
    // behind the stages: the epilogue's buffers, then the plan
    uint8_t* const epi_mem = smem + a.stages * stage_bytes;
    const PlanShared plan = plan_at(reinterpret_cast<int*>(epi_mem + epi_groups(kPair) * epi_bytes(kPair)), a.plan.E);
    volatile int* abort = &abort_s;
    // (the next kernel may be scheduled: it waits for this one before it
    // touches memory)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (tid == 0) {
        abort_s = 0;
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kPair ? 8 : 4);
        }
        mbar_init(&drained, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&part_full[i], 1);
            mbar_init(&part_empty[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_take<kPair>(&tmem_base_s);
        tc_fence_before();
    }
    plan_scan(a.plan, plan);  // ends in a block barrier
    if constexpr (kPair) cluster_sync();  // the other CTA's barriers are set up
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int nbt = mx4_nb(a.N), nbu = kPair ? (nbt + 1) / 2 : nbt, total = plan.tile[a.plan.E] * nbu;
    const int workers = gridDim.x / (kPair ? 2 : 1);

    Sched s;
    s.units = total;
    s.kb = mx4_kb(a.K);
    s.cta = blockIdx.x / (kPair ? 2 : 1);
    s.nbu = nbu;
    s.rank = rank;
    s.grid = workers;
    s.cut = cut_pays(total, s.kb, nt, workers);
    auto stage_at = [&](int st) { return smem + st * stage_bytes; };
    auto give_up = [&] {
        *abort = 1;
        if (a.status) atomicExch(a.status, static_cast<int>(MOEQ_ERR_TIMEOUT));
    };

    if (warp == 0 || warp == 2) {
        // -------------------------------------------------------- copies
        // Warp 0 copies weights, warp 2 tokens: a copy takes its thread about
        // 100 cycles, four a stage would keep the tensor cores waiting.
        if (elect_one()) {
            // weights that one token tile reads are not read again; those of
            // several, and the token tiles, come from L2 the next time
            const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
            auto weights = [&](const Part& p, int kb, int st) {
                // (an odd last block has no partner: its pair reads it twice and stores it once)
                const int64_t tile = (static_cast<int64_t>(p.e) * nbt + min(p.nb, nbt - 1)) * s.kb + kb;
                const uint64_t policy = p.tiles > 1 ? again : once;
                uint8_t* const at = stage_at(st);
                if constexpr (kPair) {
                    // both CTAs' copies count on the first's barrier
                    if (rank == 0)
                        mbar_arrive_expect_tx(
                            &full[st], 2 * (kMx4TileBytes + kMx4TileScaleBytes + p.n_mma / 2 * 128 + sfb_bytes));
                    rows_load(at, &maps.w, static_cast<int>(tile * 128), in_first(&full[st]), policy);
                    rows_load(at + off_sfa, &maps.sw, static_cast<int>(tile * 8), in_first(&full[st]), policy);
                } else {
                    mbar_arrive_expect_tx(&full[st], kMx4TileBytes + kMx4TileScaleBytes + p.n_mma * 128 + sfb_bytes);
                    bulk_load(at, a.w + tile * kMx4TileBytes, kMx4TileBytes, &full[st], policy);
                    bulk_load(at + off_sfa, a.sw + tile * kMx4TileScaleBytes, kMx4TileScaleBytes, &full[st], policy);
                }
            };
            auto tokens = [&](const Part& p, int kb, int st) {
                const int64_t block = static_cast<int64_t>(p.tile) * s.kb + kb;
                uint8_t* const at = stage_at(st);
                if constexpr (kPair) {
                    // a pair's CTAs hold half the rows each, and all the scales
                    const int half = p.n_mma / 2;
                    rows_load(at + off_b, &maps.a[half / 16 - 1], static_cast<int>(block * nt) + rank * half,
                              in_first(&full[st]), again);
                    rows_load(at + off_sfb, &maps.sa, static_cast<int>(block * (sfb_bytes / 128)), in_first(&full[st]), again);
                } else {
                    bulk_load(at + off_b, a.a + block * nt * 128, p.n_mma * 128, &full[st], again);
                    bulk_load(at + off_sfb, a.sa + block * sfb_bytes, sfb_bytes, &full[st], again);
                }
            };
            // The token tiles are written by the kernel ahead; the weights are not.
            if (warp == 2) pdl_wait();
            Part p;
            int it = 0, st = 0;
            uint32_t phase = 1;  // of the ring's previous round
            bool ok = true;
            for (int i = 0; ok && part_at(s, a, plan, i, p); ++i)
                for (int kb = p.kb0; kb < p.kb1; ++kb, ++it) {
                    if (it >= a.stages) ok = mbar_wait_bounded(&empty[st], phase, abort);
                    if (!ok) break;
                    if (warp == 0)
                        weights(p, kb, st);
                    else
                        tokens(p, kb, st);
                    if (++st == a.stages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            if (!ok) {
                give_up();
                // copies in flight land before the CTA may end (a pair's are all
                // counted in the first, and the pair ends together)
                const unsigned long long t0 = global_timer_ns();
                for (int j = max(0, it - a.stages); rank == 0 && j < it; ++j) drain(&full[j % a.stages], (j / a.stages) & 1, t0);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMAs
        // The tensor core's queue holds little, so this thread does nothing but
        // issue: the parts come ready from warp 3, and the next stage's barrier
        // is asked for while this one's last MMAs go out.
        if (rank == 0 && elect_one()) {
            const uint32_t base = smem_u32(smem) >> 4, pitch = static_cast<uint32_t>(stage_bytes) >> 4;
            const uint64_t da = umma_desc_sw128(0), db = da + (off_b >> 4);
            const uint64_t dfa = sf_desc(0) + (off_sfa >> 4), dfb = sf_desc(0) + (off_sfb >> 4);
            const uint32_t chunk = static_cast<uint32_t>(sfb_chunk) >> 4;
            int st = 0;
            uint32_t phase = 0, at = base;
            bool ok = true, ready = false;
            for (int i = 0;; ++i) {
                ok = mbar_wait_bounded(&part_full[i & 3], (i >> 2) & 1, abort);
                if (!ok) break;
                const int part = *reinterpret_cast<volatile int*>(&part_ring[i & 3]);
                mbar_arrive(&part_empty[i & 3]);
                if (!part) break;
                const int n_mma = part & 0xFFF, stages = part >> 12, buf = i & 1;
                if (i >= 2) {
                    const uint32_t ph = ((i >> 1) - 1) & 1;
                    ok = kPair ? cluster_wait_bounded(&acc_empty[buf], ph, abort) : mbar_wait_bounded(&acc_empty[buf], ph, abort);
                }
                const uint32_t d = tmem + buf * kAcc1;
                const uint32_t id0 = idesc_mx4(kPair ? 256 : 128, n_mma, 0), id2 = idesc_mx4(kPair ? 256 : 128, n_mma, 2);
                const bool wide = n_mma > 128;
                for (int k = 0; ok && k < stages; ++k) {
                    if (!ready)
                        ok = kPair ? cluster_wait_bounded(&full[st], phase, abort) : mbar_wait_bounded(&full[st], phase, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = da + at, bd = db + at, fa = dfa + at, fb = dfb + at;
                    sf_copy<kPair>(tmem + kColSfa, fa);
                    sf_copy<kPair>(tmem + kColSfb, fb);
                    if (wide) sf_copy<kPair>(tmem + kColSfb + 4, fb + (512 >> 4));
                    sf_copy<kPair>(tmem + kColSfa + 4, fa + (512 >> 4));
                    sf_copy<kPair>(tmem + kColSfb + 8, fb + chunk);
                    if (wide) sf_copy<kPair>(tmem + kColSfb + 12, fb + chunk + (512 >> 4));
                    // 64 columns = 32 bytes of a row an MMA
                    mma_mx4<kPair>(d, ad, bd, id0, tmem + kColSfa, tmem + kColSfb, k > 0);
                    mma_mx4<kPair>(d, ad + 2, bd + 2, id2, tmem + kColSfa, tmem + kColSfb, 1);
                    uint64_t* const done = &empty[st];
                    at += pitch;
                    if (++st == a.stages) {
                        st = 0;
                        phase ^= 1;
                        at = base;
                    }
                    ready = mbar_test_wait<kPair>(&full[st], phase);
                    mma_mx4<kPair>(d, ad + 4, bd + 4, id0, tmem + kColSfa + 4, tmem + kColSfb + 8, 1);
                    mma_mx4<kPair>(d, ad + 6, bd + 6, id2, tmem + kColSfa + 4, tmem + kColSfb + 8, 1);
                    mma_commit<kPair>(done);
                }
                if (!ok) break;
                mma_commit<kPair>(&acc_full[buf]);
            }
            if (!ok) {
                give_up();
                mma_commit<kPair>(&drained);
                drain(&drained, 0, global_timer_ns());
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------- parts, for the MMA thread
        if (rank == 0 && elect_one()) {
            Part p;
            bool more = true, ok = true;
            for (int i = 0; ok && more; ++i) {
                more = part_at(s, a, plan, i, p);
                if (i >= 4) ok = mbar_wait_bounded(&part_empty[i & 3], ((i >> 2) - 1) & 1, abort);
                if (!ok) break;
                *reinterpret_cast<volatile int*>(&part_ring[i & 3]) = more ? p.n_mma | (p.kb1 - p.kb0) << 12 : 0;
                mbar_arrive(&part_full[i & 3]);
            }
            if (!ok) give_up();
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------- epilogue
        pdl_wait();
        constexpr int kGroups = epi_groups(kPair);
        const int q = warp & 3, group = (warp >> 2) - 1, bar = 1 + group;
        const bool chief = tid == 128 + group * 128;
        uint8_t* stage_y = epi_mem + group * epi_bytes(kPair);
        // rows of y in 16-byte pieces
        const bool vec_y = a.N % (kF32 ? 4 : 8) == 0 && a.ld_y % (kF32 ? 4 : 8) == 0 &&
                           (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
        Part p;
        for (int i = group; part_at(s, a, plan, i, p); i += kGroups) {
            const int buf = i & 1, turn = i / kGroups & 1;
            if (lane == 0 && !mbar_wait_bounded(&acc_full[buf], (i >> 1) & 1, abort)) give_up();
            __syncwarp();
            // One thread decides for all four warps whether to go on: they meet
            // at barriers below.  (A copy a turn: a slow warp may still read the
            // last unit's.)
            if (chief) go_s[group][turn] = !*abort;
            named_sync(bar, 128);
            if (!go_s[group][turn]) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * kAcc1 + (static_cast<uint32_t>(q * 32) << 16);
            const int n = p.n0 + q * 32 + lane;
            bool join = false;  // every other part is in the workspace: this CTA adds them up
            // parts lie [unit][CTA of the pair][part], a row's columns in fours
            const size_t part_floats = static_cast<size_t>(nt) * 128;
            const int first = (kPair ? 2 * p.u + rank : p.u) * kCut, own = s.cta % kCut;
            float* const parts = a.part + first * part_floats + (q * 32 + lane) * 4;
            if (s.cut) {
                int* const ticket = a.tickets + first / kCut;
                if (chief) last_s[group][turn] = ld_acquire(ticket) == kCut - 1;
                named_sync(bar, 128);
                join = last_s[group][turn];
                if (!join) {
                    float4* slot = reinterpret_cast<float4*>(parts + own * part_floats);
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
                    named_sync(bar, 128);
                    if (chief) last_s[group][turn] = atom_add_acq_rel(ticket, 1) == kCut - 1;
                    named_sync(bar, 128);
                    join = last_s[group][turn];
                }
                if (join) {
                    __threadfence();
                    if (chief) *ticket = 0;
                }
            }
            auto release = [&] {  // the accumulator is read: the next unit but one may have it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair && rank == 1)
                        arrive_first(&acc_empty[buf]);
                    else
                        mbar_arrive(&acc_empty[buf]);
                }
            };
            if (!s.cut) {
                constexpr int kCols = epi_cols(kF32, kPair);
                for (int c0 = 0; c0 < p.n; c0 += kCols) {
                    float v[kCols];  // columns past the tile's are read and not stored
#pragma unroll
                    for (int j = 0; j < kCols; j += 16) tmem_ld16(acc + c0 + j, v + j);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < kCols; j += 16) tmem_use16(v + j);
                    if (c0 + kCols >= p.n) release();
                    store_step<kF32, kCols>(a, p, c0, q, lane, n, v, stage_y, vec_y, bar);
                }
            } else {
                for (int c0 = 0; join && c0 < p.n; c0 += 16) {
                    float v[16];
                    tmem_ld16(acc + c0, v);
                    tmem_wait_ld();
                    tmem_use16(v);
                    sum_parts(parts, part_floats, own, c0, v);
                    store_step<kF32, 16>(a, p, c0, q, lane, n, v, stage_y, vec_y, bar);
                }
                release();
            }
        }
        // rows that belong to no expert
        const int t = tid - 128;
        for (int64_t r = static_cast<int64_t>(plan.first[a.plan.E]) + blockIdx.x; r < a.plan.R; r += gridDim.x)
            for (int c = t; c < a.N; c += 128 * kGroups) store_y<kF32>(a.y, r * a.ld_y + c, 0.f);
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    if constexpr (kPair) cluster_sync();  // neither CTA's shared memory or TMEM is in use any more
    if (warp == 1) {
        tc_fence_after();
        tmem_give<kPair>(tmem);
    }
}

}  // namespace

// Rows of a token tile, and whether pairs of CTAs multiply it.  About twice
// the average of an expert, so that most experts are one tile (its weights
// then stream once), but no wider than that: a narrow tile leaves shared
// memory to more weight stages in flight.
Mx4Tiling mx4_tiling(int R, int E) {
    const long long want = E == 1 ? R : 2LL * R / E + 16;
    const bool pair = want >= kPairRows && R >= kPairRows;
    const int align = pair ? 32 : 16, most = pair ? kPairTileRows : kSingleTileRows;
    auto up = [&](long long x) { return static_cast<int>(x > most ? most : (x + align - 1) / align * align); };
    return {up(want < R ? want : R), align};
}

namespace {

bool rows_map(CUtensorMap* map, const void* p, int64_t rows, int box_rows) {
    const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(rows)}, strides[1] = {128};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, steps[2] = {1, 1};
    const EncodeTiled f = encode_tiled();
    return f && f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kF32, bool kPair>
cudaError_t launch_one(const Mx4GemmArgs& a, const typename MapsOf<kPair>::type& maps, int grid, int smem, int most_smem,
                       bool pdl, cudaStream_t stream) {
    const auto kern = mx4_gemm_kernel<kF32, kPair>;
    static OncePerDevice once;
    const cudaError_t e = raise_smem(once, reinterpret_cast<const void*>(kern), most_smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads_of(kPair));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = kPair ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, maps);
}

}  // namespace

cudaError_t launch_mx4_gemm(Mx4GemmArgs a, int grid, bool pdl, cudaStream_t stream) {
    const bool pair = a.plan.align == 32;
    const int sb = stage_bytes_of(a.plan.nt, pair);
    // of 227 KiB: less the static arrays; the stages share the rest with the
    // alignment, the epilogue's buffers and the plan
    constexpr int kMost = 227 * 1024 - 1024;
    const int rest = 1024 + epi_bytes(pair) * epi_groups(pair) + plan_ints(a.plan.E) * static_cast<int>(sizeof(int));
    const int fit = (kMost - rest) / sb;
    a.stages = fit < kMaxStages ? fit : kMaxStages;
    const int smem = a.stages * sb + rest, most = kMost;
    if (!pair)
        return a.y_f32 ? launch_one<true, false>(a, NoMaps{}, grid, smem, most, pdl, stream)
                       : launch_one<false, false>(a, NoMaps{}, grid, smem, most, pdl, stream);
    PairMaps maps;
    const int64_t tiles = static_cast<int64_t>(a.plan.E) * mx4_nb(a.N) * mx4_kb(a.K);
    const int64_t blocks = mx4_max_tiles(a.plan.R, a.plan.E, a.plan.nt) * mx4_kb(a.K);
    const int sfb_rows = mx4_tile_scale_bytes(a.plan.nt) / 128;
    if (!rows_map(&maps.w, a.w, tiles * 128, 128) || !rows_map(&maps.sw, a.sw, tiles * 8, 8) ||
        !rows_map(&maps.sa, a.sa, blocks * sfb_rows, sfb_rows))
        return cudaErrorInvalidValue;
    for (int i = 0; i < kPairTileRows / 2 / 16; ++i)
        if (!rows_map(&maps.a[i], a.a, blocks * a.plan.nt, 16 * (i + 1))) return cudaErrorInvalidValue;
    grid = grid / 2 * 2;
    return a.y_f32 ? launch_one<true, true>(a, maps, grid, smem, most, pdl, stream)
                   : launch_one<false, true>(a, maps, grid, smem, most, pdl, stream);
}

}  // namespace moeq
