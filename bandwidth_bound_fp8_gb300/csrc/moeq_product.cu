// The experts' products with bf16 weights, for rows sorted by expert, on the
// tcgen05 tensor cores (kind::f16, fp32 accumulation), in three directions:
//   y[r]  = W[e] x[r]                 product_rows_kernel, contraction over K
//   dx[r] = W[e]^T dy[r]              product_rows_kernel, contraction over N
//   dW[e] = sum_r dy[r] x[r]^T        product_weights_kernel, over e's rows
// No operand is transposed in memory: the shared-memory tiles are what lies
// there, and the MMA takes either major order.
//
// Rows out (y, dx): the weights' side is the MMA's 128-row operand (256 for a
// pair of CTAs) and the rows are its N operand, so one row an expert wastes no
// tensor time on padding.  A unit is (expert, features of a CTA or a pair, a
// tile of the expert's rows); its contraction runs in stages of 64 columns.
//   warps 0, 2  tensor copies: weights; rows
//   warp 1      issues the MMAs (one thread); warp 3 tells it the parts
//   warps 4..   epilogue: TMEM -> rows, behind the next unit's MMAs (two
//               accumulators)
// Whole units, round robin over the CTAs (pairs); none waits for another.  A
// few units are split along their contraction instead (see how_of).
//
// Weights out (dW): a unit is (expert, 256 x 256 of dW, or 256 x 128 where units
// are few) for a pair, the contraction over the expert's rows in stages of 64.
// Rows are sorted, so a stage may reach past the expert's last row: what follows
// are another expert's rows (or a NaN in a masked place), and 0 * NaN is not 0.
// So the last stage is copied row-exactly, in boxes of a power of two of rows,
// and filled up to the MMA's 16 rows with zeros.
#include "moeq_mx4_plan.cuh"
#include "moeq_pair.cuh"
#include "moeq_rows.h"

namespace moeq {
namespace {

constexpr int kBlock = 64;                      // contraction a stage: 128 bytes of bf16, the swizzle's span
constexpr int kTileBytes = 128 * kBlock * 2;    // 128 features (or dW rows / columns) of a stage
constexpr int kAcc1 = 256;                      // TMEM columns of the second accumulator
// Stages in flight at most.  More gain a little where few CTAs have a long
// contraction and lose elsewhere; us with 5, 7, 9 and 12: one token over 8 of 256
// experts (K 6144, N 4096) 67.5, 65.1, 64.0 and 63.6; 6 rows each of 256 experts
// (K 2048, N 2816) 427, 418, 424 and 422, their gradient 418, 407, 426 and 426.
constexpr int kMaxStages = 7;
// Most rows of a tile, for one CTA and for a pair.
constexpr int kSingleTileRows = 128, kPairTileRows = 256;
// Tiles of this many rows are a pair's.  An average of 72 or 100 rows an expert
// (64 of them, sizes spread by a fifth) takes pairs 1 to 2 % longer than single
// CTAs, 128 rows 4 to 8 % less, 256 rows a quarter less.
constexpr int kPairRows = 128;
// Steps of 16 contraction indices that one accumulator takes where the output
// is fp32: the tensor core truncates as it accumulates, so parts of 512 are
// summed in registers (over K = 2048 the error against 64 bits is 5.1e-7 of the
// result, with one accumulator 2.6e-6; a plain fp32 product's is 5e-7).
constexpr int kRun = 32;
// The same where it is bf16: parts of 1024.  An accumulator of the whole
// contraction tips roundings: of 6144, 0.35 % of the values of y are not the
// exact sum's nearest, of 65536 terms of one sign 3 %; so 0.07 % at any length
// (with parts of 512 0.04 %).  The parts cost 0 to 1.4 % (64 experts of 384
// rows, 6144 -> 4096: 803 us whole, 811 so, 825 in parts of 512).  And no thread
// waits long for one part of a sum over millions of rows.
constexpr int kBf16Run = 64;
// Row tiles that take turns on the same weights, so that a wave of CTAs covers
// a block of both operands: a dense product of 16384 rows (6144 -> 4096) takes
// 437 us so, and 503 with all 64 tiles in a row.
constexpr int kBand = 8;

// A stage: the weights' tile, then the rows' tile.  A box that would pass the
// matrix's last row is slow (one row for each of 8 experts, 1408 x 2048: 11.8 us
// with it, 9.7 without), so a single CTA's starts earlier there, and the rows
// ahead of the tile's first land in front of the tile: up to 15.
__host__ __device__ constexpr int rows_at(bool pair) { return kTileBytes + (pair ? 0 : 2048); }
__host__ __device__ constexpr int stage_bytes_of(int nt, bool pair) { return rows_at(pair) + nt / (pair ? 2 : 1) * 128; }

// ------------------------------------------------------------- instructions
// A and B bf16, D fp32, m x n; a_mn, b_mn: the operand's M (N) index is the
// one that runs along memory.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
template <bool kPair>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int acc) {
    if constexpr (kPair)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
// An operand whose M (N) index runs along memory, 128-byte swizzle: columns of
// 64 of it, kBlock rows of 128 bytes each (one a contraction index), one after
// the other.  The next 16 contraction indices are 2048 bytes on.
__device__ __forceinline__ uint64_t desc_mn(uint32_t smem_addr) {
    uint64_t d = static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kBlock * 128 >> 4) << 16;  // to the next 64
    d |= static_cast<uint64_t>(1024 >> 4) << 32;          // to the next 8 contraction indices
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
// A box into this CTA's shared memory, counted on `bar` (an address in the
// cluster: a pair's copies count on the first CTA's).
template <bool kPair>
__device__ __forceinline__ void copy2(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t policy) {
    if constexpr (kPair)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
            : "memory");
}
template <bool kPair>
__device__ __forceinline__ void copy3(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                      uint64_t policy) {
    if constexpr (kPair)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
            : "memory");
}
// Two neighbouring columns of 64 at once, of a matrix whose rows are whole
// columns; they lie one after the other in shared memory.
__device__ __forceinline__ void copy_columns(void* dst, const CUtensorMap* map, int col, int row, uint32_t bar,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(col / kBlock), "r"(bar), "l"(policy)
        : "memory");
}
// A box out of shared memory.
__device__ __forceinline__ void store3(const CUtensorMap* map, const void* src, int x, int y, int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2, %3}], [%4], %5;" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(x), "r"(y), "r"(z), "r"(smem_u32(src)), "l"(policy)
        : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// What this thread wrote to shared memory, for copies that it or (behind a
// barrier) another starts.
__device__ __forceinline__ void fence_smem_for_copies() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t part_of(int n, int steps) {
    return static_cast<uint32_t>(steps) << 5 | static_cast<uint32_t>(n >> 4);
}
// A map's fetch from memory is then behind its first copy.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Barriers and the queue of parts that both kernels have.
struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
    uint64_t part_full[4], part_empty[4];
    uint64_t joined;  // the other CTAs' sums of a unit whose contraction is split
    uint32_t part_ring[4], tmem_base;
    int abort, go[2][2];
};

// Set-up up to the point where memory may be read.  (TMEM is taken ahead of the
// wait for the kernel before: the library's kernels that use it hold 36000
// registers or more a CTA, so no two of them share an SM, and none waits here
// for columns that a later one holds.)  Ends in a block barrier
// (plan_scan's) and, for a pair or a split, one of the cluster.
template <bool kPair, bool kSplit>
__device__ __forceinline__ uint32_t set_up(Shared& s, int stages, int split, const Mx4Plan& p, const PlanShared& plan) {
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        s.abort = 0;
        for (int i = 0; i < stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], kPair ? 16 : 4);  // every epilogue warp of both CTAs
        }
        mbar_init(&s.drained, 1);
        if (kSplit) mbar_init(&s.joined, 4 * (split - 1));
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s.part_full[i], 1);
            mbar_init(&s.part_empty[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_take<kPair>(&s.tmem_base);
        tc_fence_before();
    }
    chain();
    plan_scan(p, plan);
    if constexpr (kPair || kSplit) cluster_sync();  // the other CTAs' barriers are set up
    tc_fence_after();
    return s.tmem_base;
}

// The ring of stages as its users walk it.
struct Ring {
    int stages, at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == stages) {
            at = 0;
            phase ^= 1;
        }
    }
};

// The thread that issues the MMAs: for each part of the queue, its stages.
// A part is part_of(N of the MMAs, how many of 16 contraction indices there
// are); 0 ends the queue.
template <bool kPair, int kStepA, int kStepB, typename Desc>
__device__ __forceinline__ void issue_parts(Shared& s, int stages, int stage_bytes, uint32_t tmem, uint64_t da, uint64_t db,
                                            Desc idesc_of, volatile int* abort, int* status) {
    const uint32_t pitch = static_cast<uint32_t>(stage_bytes) >> 4;
    Ring ring{stages};
    uint32_t at = 0;
    bool ok = true, ready = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return kPair ? cluster_wait_bounded(bar, parity, abort) : mbar_wait_bounded(bar, parity, abort);
    };
    for (int i = 0;; ++i) {
        ok = mbar_wait_bounded(&s.part_full[i & 3], (i >> 2) & 1, abort);
        if (!ok) break;
        const uint32_t part = *reinterpret_cast<volatile uint32_t*>(&s.part_ring[i & 3]);
        mbar_arrive(&s.part_empty[i & 3]);
        if (!part) break;
        const int buf = i & 1;
        int steps = static_cast<int>(part >> 5);
        if (i >= 2) ok = wait(&s.acc_empty[buf], ((i >> 1) - 1) & 1);
        const uint32_t d = tmem + buf * kAcc1, id = idesc_of(static_cast<int>(part & 31) << 4);
        for (int k = 0; ok && steps > 0; ++k, steps -= 4) {
            if (!ready) ok = wait(&s.full[ring.at], ring.phase);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = da + at, b = db + at;
            mma_bf16<kPair>(d, a, b, id, k > 0);
            if (steps > 1) mma_bf16<kPair>(d, a + kStepA, b + kStepB, id, 1);
            uint64_t* const done = &s.empty[ring.at];
            ring.next();
            at = ring.at * pitch;
            ready = mbar_test_wait<kPair>(&s.full[ring.at], ring.phase);
            if (steps > 2) mma_bf16<kPair>(d, a + 2 * kStepA, b + 2 * kStepB, id, 1);
            if (steps > 3) mma_bf16<kPair>(d, a + 3 * kStepA, b + 3 * kStepB, id, 1);
            mma_commit<kPair>(done);
        }
        if (!ok) break;
        mma_commit<kPair>(&s.acc_full[buf]);
    }
    if (!ok) {
        *abort = 1;
        if (status) atomicExch(status, static_cast<int>(MOEQ_ERR_TIMEOUT));
        mma_commit<kPair>(&s.drained);
        drain(&s.drained, 0, global_timer_ns());
    }
}

// Puts a part into the queue; false where the wait for room gave up.
__device__ __forceinline__ bool push_part(Shared& s, int i, uint32_t part, volatile int* abort) {
    if (i >= 4 && !mbar_wait_bounded(&s.part_empty[i & 3], ((i >> 2) - 1) & 1, abort)) return false;
    *reinterpret_cast<volatile uint32_t*>(&s.part_ring[i & 3]) = part;
    mbar_arrive(&s.part_full[i & 3]);
    return true;
}

// Whether the four warps of an epilogue group go on to a part whose
// accumulator they wait for: one thread decides for all, because they meet at
// barriers.  (A copy a turn: a slow warp may still read the last part's.)
template <typename GiveUp>
__device__ __forceinline__ bool part_done(Shared& s, int i, int group, int lane, bool chief, volatile int* abort,
                                          GiveUp give_up) {
    if (lane == 0 && !mbar_wait_bounded(&s.acc_full[i & 1], (i >> 1) & 1, abort)) give_up();
    __syncwarp();
    if (chief) s.go[group][i & 1] = !*abort;
    named_sync(1 + group, 128);
    if (!s.go[group][i & 1]) return false;
    tc_fence_after();
    return true;
}
// The accumulator is read: the next part but one may have it.  The arrival at
// the other CTA's barrier is relaxed: the fence orders the accumulator, and a
// release to the cluster would wait for this thread's stores of the part
// before (1.2 us: 954 us where dW's stores alone take 554).
template <bool kPair>
__device__ __forceinline__ void release_acc(Shared& s, int buf, int rank, int lane) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
        if (kPair && rank == 1)
            asm volatile(
                "{ .reg .b32 r; mapa.shared::cluster.u32 r, %0, 0;\n"
                "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [r]; }" ::"r"(smem_u32(&s.acc_empty[buf]))
                : "memory");
        else
            mbar_arrive(&s.acc_empty[buf]);
    }
}
// A part's `cols` columns (at most kA kB) of this thread's lane into registers,
// or added to what is there; then the accumulator is free.  All loads of a
// first part are in flight at once: the MMAs of the part after next wait for
// them.
template <bool kPair, int kA, int kB>
__device__ __forceinline__ void take_acc(Shared& s, int buf, uint32_t acc, int cols, bool first, int rank, int lane,
                                         float (&v)[kA][kB]) {
    static_assert(kB % 16 == 0, "loads of 16 columns");
    if (first) {
#pragma unroll
        for (int c = 0; c < kA * kB; c += 16)
            if (c < cols) tmem_ld16(acc + c, v[c / kB] + c % kB);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kA * kB; c += 16) tmem_use16(v[c / kB] + c % kB);
    } else {
#pragma unroll
        for (int c = 0; c < kA * kB; c += 16)
            if (c < cols) {
                float t[16];
                tmem_ld16(acc + c, t);
                tmem_wait_ld();
                tmem_use16(t);
#pragma unroll
                for (int k = 0; k < 16; ++k) v[c / kB][c % kB + k] += t[k];
            }
    }
    release_acc<kPair>(s, buf, rank, lane);
}

// A unit whose contraction is split over a cluster: every CTA but the first
// leaves its sums in the first's shared memory ([CTA][column][lane]), and the
// first adds them to its own in the order of the contraction.
template <int kA, int kB>
__device__ __forceinline__ void send_sums(Shared& s, const float* join, int part_floats, int rank, int q, int cols,
                                          int lane, const float (&v)[kA][kB]) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                 : "=r"(at)
                 : "r"(smem_u32(join + (rank - 1) * part_floats + q * 32 + lane)));
#pragma unroll
    for (int c = 0; c < 128; ++c)
        if (c < cols) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + c * 512), "f"(v[c / kB][c % kB]) : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    __syncwarp();
    if (lane == 0) arrive_first(&s.joined);
}
template <int kA, int kB, typename GiveUp>
__device__ __forceinline__ bool add_sums(Shared& s, const float* join, int part_floats, int split, int q, int cols,
                                         int lane, bool chief, volatile int* abort, GiveUp give_up, float (&v)[kA][kB]) {
    if (lane == 0 && !cluster_wait_bounded(&s.joined, 0, abort)) give_up();
    __syncwarp();
    if (chief) s.go[1][0] = !*abort;
    named_sync(1, 128);
    if (!s.go[1][0]) return false;
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    for (int r = 1; r < split; ++r, join += part_floats)
#pragma unroll
        for (int c = 0; c < 128; ++c)
            if (c < cols) v[c / kB][c % kB] += join[c * 128 + q * 32 + lane];
    return true;
}

// A pair's 384 threads start with 168 registers each; the epilogue's 256 take
// 40 more from the 128 that copy and issue: 128 * 88 + 256 * 208 = 384 * 168.
template <bool kPair>
__device__ __forceinline__ void give_registers() {
    if constexpr (kPair) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
}
template <bool kPair>
__device__ __forceinline__ void take_registers() {
    if constexpr (kPair) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
}

// ----------------------------------------------------------------- rows out
struct RowsArgs {
    Mx4Plan plan;
    void* y;
    int64_t ld_y;
    int N, C;  // features of a row of y, contraction
    int stages;
    int split;  // CTAs (a cluster) that share a unit's contraction
    int* status;
};
struct RowsMaps {
    CUtensorMap w;
    CUtensorMap x[kSingleTileRows / 16];  // 16 rows, 32, ... (a pair's CTA copies half a tile)
};

struct Part {
    int n0, r0, n, n_mma, tiles, e;
};
// The i-th part of this CTA (pair); false past its last.  Units count experts,
// then bands of kBand row tiles, then blocks of features, then the band's
// tiles: CTAs at work together share both operands in L2, whatever the
// expert's size.
template <bool kPair>
__device__ __forceinline__ bool part_at(const RowsArgs& a, const PlanShared& plan, int i, int worker, int workers,
                                        int nbu, int rank, Part& p) {
    const int u = worker + i * workers;
    if (u >= plan.tile[a.plan.E] * nbu) return false;
    const int e = plan_find(plan.tile, a.plan.E, u / nbu);  // experts without tiles are never the last such
    const int r0 = plan.first[e], cnt = plan.first[e + 1] - r0;
    const int tiles = plan.tile[e + 1] - plan.tile[e], per = plan_rows_per_tile(cnt, a.plan.nt, a.plan.align);
    const int local = u - plan.tile[e] * nbu, band = local / (nbu * kBand), in = local - band * nbu * kBand;
    const int width = min(kBand, tiles - band * kBand), nb = in / width, t = band * kBand + in - nb * width;
    p.e = e;
    p.tiles = tiles;
    p.n0 = (kPair ? 2 * nb + rank : nb) * 128;
    p.r0 = r0 + t * per;
    p.n = min(per, cnt - t * per);
    p.n_mma = (p.n + a.plan.align - 1) & ~(a.plan.align - 1);
    return true;
}

// kSplit (of single CTAs): a cluster has one unit, and each of its CTAs a share
// of the contraction.
template <bool kF32, bool kPair, bool kTrans, bool kSplit>
__global__ void __launch_bounds__(threads_of(kPair), 1)
    product_rows_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ RowsMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared s;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int stage_bytes = stage_bytes_of(a.plan.nt, kPair);
    const int rank = kPair ? static_cast<int>(cluster_rank()) : 0;
    const int split = kSplit ? a.split : 1, srank = kSplit ? static_cast<int>(cluster_rank()) : 0;
    // behind the stages: the others' sums, the epilogue's buffers, the plan
    float* const join = reinterpret_cast<float*>(smem + a.stages * stage_bytes);
    const int part_floats = a.plan.nt * 128;
    uint8_t* const epi_mem = reinterpret_cast<uint8_t*>(join + (split - 1) * part_floats);
    const PlanShared plan = plan_at(reinterpret_cast<int*>(epi_mem + epi_groups(kPair) * epi_bytes(kPair)), a.plan.E);
    if (tid == 0) prefetch_map(&maps.w);
    if (tid == 64) prefetch_map(&maps.x[a.plan.nt / (kPair ? 32 : 16) - 1]);
    const uint32_t tmem = set_up<kPair, kSplit>(s, a.stages, split, a.plan, plan);
    volatile int* abort = &s.abort;
    const int each = kPair ? 2 : split, workers = gridDim.x / each, worker = blockIdx.x / each;
    const int nbu = kPair ? (a.N + 255) / 256 : (a.N + 127) / 128, kb_n = (a.C + kBlock - 1) / kBlock;
    const int kb0 = kb_n * srank / split, kb1 = kb_n * (srank + 1) / split;  // (kb_n * 8 < 2^18)
    const int steps_n = 4 * (kb1 - kb0), run = kF32 ? kRun : kBf16Run;       // of 16; a part's
    auto part = [&](int i, Part& p) {
        return (!kSplit || i == 0) && part_at<kPair>(a, plan, i, worker, workers, nbu, rank, p);
    };
    auto give_up = [&] {
        *abort = 1;
        if (a.status) atomicExch(a.status, static_cast<int>(MOEQ_ERR_TIMEOUT));
    };

    if (warp < 4) give_registers<kPair>();
    if (warp == 0 || warp == 2) {
        // -------------------------------------------------------- copies
        if (elect_one()) {
            // weights that one tile reads are not read again; those of several,
            // and the rows, come from L2 the next time
            const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
            Part p;
            Ring ring{a.stages};
            int it = 0;
            bool ok = true;
            for (int i = 0; ok && part(i, p); ++i)
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    if (it >= a.stages) ok = mbar_wait_bounded(&s.empty[ring.at], ring.phase ^ 1, abort);
                    if (!ok) break;
                    uint8_t* const at = smem + ring.at * stage_bytes;
                    const uint32_t bar = kPair ? in_first(&s.full[ring.at]) : smem_u32(&s.full[ring.at]);
                    const int rows = kPair ? p.n_mma / 2 : min(p.n_mma, a.plan.R);  // of the box
                    if (warp == 0) {
                        // both CTAs' copies of a pair count on the first's barrier
                        if (rank == 0)
                            mbar_arrive_expect_tx(&s.full[ring.at], (kPair ? 2 : 1) * (kTileBytes + rows * 128));
                        const uint64_t policy = p.tiles > 1 ? again : once;
                        if constexpr (kTrans) {
                            copy3<kPair>(at, &maps.w, p.n0, kb * kBlock, p.e, bar, policy);
                            copy3<kPair>(at + kTileBytes / 2, &maps.w, p.n0 + 64, kb * kBlock, p.e, bar, policy);
                        } else {
                            copy3<kPair>(at, &maps.w, kb * kBlock, p.n0, p.e, bar, policy);
                        }
                    } else {
                        const int from = kPair ? p.r0 + rank * rows : min(p.r0, a.plan.R - rows);
                        uint8_t* const to = at + rows_at(kPair) - (kPair ? 0 : (p.r0 - from) * 128);
                        copy2<kPair>(to, &maps.x[p.n_mma / (kPair ? 32 : 16) - 1], kb * kBlock, from, bar, again);
                    }
                    ring.next();
                }
            if (!ok) {
                give_up();
                // copies in flight land before the CTA may end (a pair's are all
                // counted in the first, and the pair ends together)
                const unsigned long long t0 = global_timer_ns();
                for (int j = max(0, it - a.stages); rank == 0 && j < it; ++j)
                    drain(&s.full[j % a.stages], (j / a.stages) & 1, t0);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMAs
        if (rank == 0 && elect_one()) {
            const uint32_t base = smem_u32(smem);
            const uint64_t da = kTrans ? desc_mn(base) : umma_desc_sw128(base), db = umma_desc_sw128(base + rows_at(kPair));
            // 16 contraction indices on: 32 bytes of a row, or 16 rows
            issue_parts<kPair, kTrans ? 128 : 2, 2>(
                s, a.stages, stage_bytes, tmem, da, db,
                [](int n) { return idesc_bf16(kPair ? 256 : 128, n, kTrans, false); }, abort, a.status);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------- parts, for the MMA thread
        if (rank == 0 && elect_one()) {
            Part p;
            bool more = true, ok = true;
            for (int u = 0, i = 0; ok && more;) {
                more = part(u++, p);
                if (!more) ok = push_part(s, i, 0, abort);
                for (int k0 = 0; ok && more && k0 < steps_n; k0 += run)
                    ok = push_part(s, i++, part_of(p.n_mma, min(run, steps_n - k0)), abort);
            }
            if (!ok) give_up();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- epilogue
        take_registers<kPair>();
        // Lane = feature.  A pair's two groups share a tile's columns.
        constexpr int kGroups = epi_groups(kPair), kCols = epi_cols(kF32, kPair);
        const int q = warp & 3, group = (warp >> 2) - 1, bar = 1 + group;
        const bool chief = tid == 128 + group * 128;
        uint8_t* stage_y = epi_mem + group * epi_bytes(kPair);
        // rows of y in 16-byte pieces
        const bool vec_y = a.N % (kF32 ? 4 : 8) == 0 && a.ld_y % (kF32 ? 4 : 8) == 0 &&
                           (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
        Part p;
        bool ok = true;
        for (int u = 0, i = 0; part(u, p); ++u) {
            const int share = kPair ? p.n_mma / 2 : p.n_mma, base = group * share, cols = min(share, p.n - base);
            float v[128 / kCols][kCols];
            for (int k0 = 0; ok && k0 < steps_n; k0 += run, ++i) {
                ok = part_done(s, i, group, lane, chief, abort, give_up);
                if (!ok) break;
                const uint32_t acc = tmem + (i & 1) * kAcc1 + base + (static_cast<uint32_t>(q * 32) << 16);
                take_acc<kPair>(s, i & 1, acc, cols, k0 == 0, rank, lane, v);
            }
            if (!ok) break;
            if constexpr (kSplit) {
                if (srank > 0) {
                    send_sums(s, join, part_floats, srank, q, cols, lane, v);
                    continue;
                }
                ok = add_sums(s, join, part_floats, split, q, cols, lane, chief, abort, give_up, v);
                if (!ok) break;
            }
            const int n = p.n0 + q * 32 + lane;
            p.n = base + cols;
#pragma unroll
            for (int c = 0; c < 128; c += kCols)
                if (c < cols) store_step<kF32, kCols>(a, p, base + c, q, lane, n, v[c / kCols], stage_y, vec_y, bar);
        }
        // rows that belong to no expert
        const int t = tid - 128, per = vec_y ? (kF32 ? 4 : 8) : 1;
        for (int64_t r = static_cast<int64_t>(plan.first[a.plan.E]) + blockIdx.x; r < a.plan.R; r += gridDim.x)
            for (int c = t * per; c < a.N; c += 128 * kGroups * per) {
                if (vec_y)
                    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.y) + (r * a.ld_y + c) * (kF32 ? 4 : 2)) =
                        make_uint4(0, 0, 0, 0);
                else
                    store_y<kF32>(a.y, r * a.ld_y + c, 0.f);
            }
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    if constexpr (kPair || kSplit) cluster_sync();  // no CTA's shared memory or TMEM is in use any more
    if (warp == 1) {
        tc_fence_after();
        tmem_give<kPair>(tmem);
    }
}

// -------------------------------------------------------------- weights out
struct WeightsArgs {
    Mx4Plan plan;
    int N, K;
    int stages;
    bool whole;  // N and K are whole columns of 64
    int* status;
};
struct WeightsMaps {
    CUtensorMap dy[7], x[7];  // 64 rows, 32, .. 1
    CUtensorMap dy2, x2;      // 64 rows of two columns of 64
    CUtensorMap dw;
};
// A unit is 256 rows of dW and kWide columns, 256 or 128 (see wide_units).
// A stage: a CTA's 128 rows, and half of the columns.
template <int kWide>
constexpr int kWStageBytes = kTileBytes + kWide / 2 * 128;
constexpr int kWEpiBytes = 8 * 4096;          // 128 bytes of 32 rows for each epilogue warp

struct WPart {
    int e, n0, k0, r0, cnt;
};
template <int kWide>
__device__ __forceinline__ bool wpart_at(const WeightsArgs& a, const PlanShared& plan, int i, int worker, int workers,
                                         WPart& p) {
    const int nbu = (a.N + 255) / 256, kbu = (a.K + kWide - 1) / kWide, u = worker + i * workers;
    if (u >= a.plan.E * nbu * kbu) return false;
    p.e = u / (nbu * kbu);
    const int in = u - p.e * nbu * kbu, nb = in / kbu;
    p.n0 = nb * 256;
    p.k0 = (in - nb * kbu) * kWide;
    p.r0 = plan.first[p.e];
    p.cnt = plan.first[p.e + 1] - p.r0;
    return true;
}

// 64 rows of two columns of 64 (or one), or fewer at the end of an expert's, into a stage.  Two
// boxes of the largest power of two cover any count, one from each end (what
// both write is the same).  (A box for each bit of the count: 64 experts of 383
// rows, K 6144, N 4096, took 1030 us where 384 take 868.)
struct Boxes {
    int m, n;  // maps[m]: 64 >> m rows; how many boxes
};
__device__ __forceinline__ Boxes boxes_of(int rows) {
    const int m = __clz(rows) - 25;  // the largest box of at most `rows` rows
    return {m, kBlock >> m == rows ? 1 : 2};
}
// The rows that arrive, those copied twice twice.
__device__ __forceinline__ int copied_rows(int rows) {
    const Boxes v = boxes_of(rows);
    return v.n * (kBlock >> v.m);
}
// The copying threads have little time, so whole stages take one copy where
// they can (maps2) and none of the arithmetic: a dense dW of 16384 rows (K 6144,
// N 4096) takes 566 us so and 612 without, 64 experts of 384 rows (K 2048, N
// 2816) 232 and 251.
__device__ __forceinline__ void copy_rows(uint8_t* at, const CUtensorMap* maps, const CUtensorMap* maps2, bool whole,
                                          bool two, int col, int r0, int rows, uint32_t bar, uint64_t policy) {
    if (rows == kBlock) {
        if (whole && two) {
            copy_columns(at, maps2, col, r0, bar, policy);
        } else {
            copy2<true>(at, &maps[0], col, r0, bar, policy);
            if (two) copy2<true>(at + kTileBytes / 2, &maps[0], col + 64, r0, bar, policy);
        }
        return;
    }
    const Boxes v = boxes_of(rows);
    for (int i = 0; i < v.n; ++i) {
        const int to = i ? rows - (kBlock >> v.m) : 0;
        copy2<true>(at + to * 128, &maps[v.m], col, r0 + to, bar, policy);
        if (two) copy2<true>(at + kTileBytes / 2 + to * 128, &maps[v.m], col + 64, r0 + to, bar, policy);
    }
}
// The rows behind them up to the next multiple of 16: zeros, written by the warp
// whose copies into the same stage follow, so that the MMAs that wait for those
// copies find them.  Nothing else orders the zeros ahead of the MMAs: every lane's
// stores are complete for the async proxy at its fence, the copies start behind
// it, and the MMA thread waits for the bytes of both CTAs' copies, of this warp's
// among them.  (An arrival of its own, released to the cluster, costs 0.4 us a
// unit.  Zeros copied from beyond the matrix, or from an array of
// them, cost more than the rows: 64 experts of 376 rows, K 6144, N 4096, 1046
// us, so 950.)
__device__ __forceinline__ void zero_rows(uint8_t* at, bool two, int rows, int lane) {
    uint8_t* const to = at + (two && (lane & 8) ? kTileBytes / 2 : 0) + (lane & 7) * 16;
    for (int r = rows + (two ? lane >> 4 : lane >> 3); r < ((rows + 15) & ~15); r += two ? 2 : 4)
        *reinterpret_cast<uint4*>(to + r * 128) = make_uint4(0, 0, 0, 0);
    fence_smem_for_copies();
    __syncwarp();
}

template <bool kF32, int kWide>
__global__ void __launch_bounds__(threads_of(true), 1)
    product_weights_kernel(const __grid_constant__ WeightsArgs a, const __grid_constant__ WeightsMaps maps) {
    // (everything is dynamic, and starts where the swizzle's pattern does: six
    // stages then fit beside the epilogue's buffers)
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_rank());
    uint8_t* const epi_mem = smem + a.stages * kWStageBytes<kWide>;
    Shared& s = *reinterpret_cast<Shared*>(epi_mem + kWEpiBytes);
    const PlanShared plan = plan_at(reinterpret_cast<int*>(&s + 1), a.plan.E);
    if (tid == 0) prefetch_map(a.whole ? &maps.dy2 : &maps.dy[0]);
    if (tid == 64) prefetch_map(a.whole ? &maps.x2 : &maps.x[0]);
    if (tid == 128) prefetch_map(&maps.dw);
    const uint32_t tmem = set_up<true, false>(s, a.stages, 1, a.plan, plan);
    volatile int* abort = &s.abort;
    const int workers = gridDim.x / 2, worker = blockIdx.x / 2;
    auto part = [&](int i, WPart& p) { return wpart_at<kWide>(a, plan, i, worker, workers, p); };
    auto give_up = [&] {
        *abort = 1;
        if (a.status) atomicExch(a.status, static_cast<int>(MOEQ_ERR_TIMEOUT));
    };

    if (warp < 4) give_registers<true>();
    if (warp == 0 || warp == 2) {
        // -------------------------------------------------------- copies
        // Warp 0 copies dy, warp 2 x: both come from L2 for every block of dW.
        const uint64_t again = l2_evict_normal_policy();
        const bool leader = elect_one();
        const CUtensorMap* const some = warp == 0 ? maps.dy : maps.x;
        const CUtensorMap* const pairs = warp == 0 ? &maps.dy2 : &maps.x2;
        const bool two = kWide == 256 || warp == 0;  // columns of 64 that this CTA copies
        uint8_t* const mine = smem + (warp == 0 ? 0 : kTileBytes);
        WPart p;
        Ring ring{a.stages};
        int it = 0;
        bool ok = true;
        for (int i = 0; ok && part(i, p); ++i) {
            const int col = (warp == 0 ? p.n0 : p.k0) + rank * (two ? 128 : 64);
            const auto copies = [&](int r, int rows) {
                // both CTAs' columns of 64 of both operands
                if (warp == 0 && rank == 0)
                    mbar_arrive_expect_tx(&s.full[ring.at], (256 + kWide) / 64 * 128 * copied_rows(rows));
                copy_rows(mine + ring.at * kWStageBytes<kWide>, some, pairs, a.whole, two, col, p.r0 + r, rows,
                          in_first(&s.full[ring.at]), again);
            };
            const int whole = p.cnt & ~(kBlock - 1), rows = p.cnt - whole;
            if (leader) {
                for (int r = 0; r < whole; r += kBlock, ++it) {
                    if (it >= a.stages) ok = mbar_wait_bounded(&s.empty[ring.at], ring.phase ^ 1, abort);
                    if (!ok) break;
                    copies(r, kBlock);
                    ring.next();
                }
                if (ok && rows && it >= a.stages) ok = mbar_wait_bounded(&s.empty[ring.at], ring.phase ^ 1, abort);
            }
            ok = __all_sync(~0u, ok);
            if (!ok || rows == 0) continue;
            if (rows & 15) {
                __syncwarp();  // what the leader waited for
                zero_rows(mine + __reduce_max_sync(~0u, leader ? ring.at : 0) * kWStageBytes<kWide>, two, rows, lane);
            }
            if (leader) {
                copies(whole, rows);
                ring.next();
                ++it;
            }
        }
        if (leader && !ok) {
            give_up();
            const unsigned long long t0 = global_timer_ns();
            for (int j = max(0, it - a.stages); rank == 0 && j < it; ++j)
                drain(&s.full[j % a.stages], (j / a.stages) & 1, t0);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMAs
        if (rank == 0 && elect_one()) {
            const uint32_t base = smem_u32(smem);
            issue_parts<true, 128, 128>(
                s, a.stages, kWStageBytes<kWide>, tmem, desc_mn(base), desc_mn(base + kTileBytes),
                [](int n) { return idesc_bf16(256, n, true, true); }, abort, a.status);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------- parts, for the MMA thread
        if (rank == 0 && elect_one()) {
            WPart p;
            bool more = true, ok = true;
            for (int u = 0, i = 0; ok && more;) {
                more = part(u++, p);
                if (!more) ok = push_part(s, i, 0, abort);
                const int steps_n = (p.cnt + 15) / 16, run = kF32 ? kRun : kBf16Run;
                for (int k0 = 0; ok && more && k0 < steps_n; k0 += run)
                    ok = push_part(s, i++, part_of(kWide, min(run, steps_n - k0)), abort);
            }
            if (!ok) give_up();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- epilogue
        take_registers<true>();
        // Lane = row of dW; the two groups share the columns, which leave
        // registers through shared memory, 128 bytes of a warp's 32 rows at a time,
        // as tensor copies (they clip at N and K).  (Stored by the lanes, 32 bytes
        // each, dW goes out at 4.1 TB/s; so at 6.8.)  An expert without rows has
        // no part: it gets zeros.
        const int q = warp & 3, group = (warp >> 2) - 1;
        const bool chief = tid == 128 + group * 128;
        uint8_t* const buf_y = epi_mem + (group * 4 + q) * (kWEpiBytes / 8);
        constexpr int kCols = kF32 ? 32 : 64, kMine = kWide / 2;  // a step's and a group's columns
        // dW is not read again here: left to stay in L2 it drives out dy and x (256
        // experts of 128 rows, K 6144, N 4096: 2550 us so, 2385 with this)
        const uint64_t once = l2_evict_first_policy();
        WPart p;
        bool ok = true;
        for (int u = 0, i = 0; part(u, p); ++u) {
            const int n0 = p.n0 + rank * 128 + q * 32, k0 = p.k0 + group * kMine;
            const int steps_n = (p.cnt + 15) / 16, run = kF32 ? kRun : kBf16Run;
            float v[kMine / kCols][kCols];
            if (p.cnt == 0) {
#pragma unroll
                for (int c = 0; c < kMine; ++c) v[c / kCols][c % kCols] = 0.f;
            }
            for (int st = 0; ok && st < steps_n; st += run, ++i) {
                ok = part_done(s, i, group, lane, chief, abort, give_up);
                if (!ok) break;
                const uint32_t acc = tmem + (i & 1) * kAcc1 + group * kMine + (static_cast<uint32_t>(q * 32) << 16);
                take_acc<true>(s, i & 1, acc, kMine, st == 0, rank, lane, v);
            }
            if (!ok) break;
#pragma unroll
            for (int c0 = 0; c0 < kMine; c0 += kCols) {
                if (n0 >= a.N || k0 + c0 >= a.K) continue;
                const float(&w)[kCols] = v[c0 / kCols];
                if (lane == 0) stores_read();  // the copy before has left the buffer
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (kF32) {
                            x[k] = __float_as_uint(w[4 * c + k]);
                        } else {
                            const __nv_bfloat162 t = __floats2bfloat162_rn(w[8 * c + 2 * k], w[8 * c + 2 * k + 1]);
                            x[k] = *reinterpret_cast<const uint32_t*>(&t);
                        }
                    }
                    *reinterpret_cast<uint4*>(buf_y + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
                }
                fence_smem_for_copies();
                __syncwarp();
                if (lane == 0) store3(&maps.dw, buf_y, k0 + c0, n0, p.e, once);
            }
        }
        if (lane == 0) stores_done();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();  // neither CTA's shared memory or TMEM is in use any more
    if (warp == 1) {
        tc_fence_after();
        tmem_give<true>(tmem);
    }
}

// --------------------------------------------------------------------- host
bool encode(CUtensorMap* map, const void* p, int dims_n, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    const EncodeTiled f = encode_tiled();
    return f && f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims_n, const_cast<void*>(p), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map2(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {kBlock, static_cast<cuuint32_t>(box_rows)};
    return encode(map, p, 2, dims, strides, box);
}
// For copy_columns: 64 rows of two columns of 64; cols is a multiple of 64.
bool columns_map(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld) {
    const cuuint64_t dims[3] = {kBlock, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / kBlock)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, kBlock * 2};
    const cuuint32_t box[3] = {kBlock, kBlock, 2};
    return encode(map, p, 3, dims, strides, box);
}
// [E, N, K], contiguous; the box is one expert's.
bool map3(CUtensorMap* map, const void* p, int f32, int64_t K, int64_t N, int64_t E, int box_k, int box_n) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(E)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K) * (f32 ? 4 : 2), static_cast<cuuint64_t>(K * N) * (f32 ? 4 : 2)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_k), static_cast<cuuint32_t>(box_n), 1}, steps[3] = {1, 1, 1};
    const EncodeTiled f = encode_tiled();
    return f && f(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p),
                  dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Args, typename Maps>
cudaError_t launch(void (*kern)(Args, Maps), OncePerDevice& once, const Args& a, const Maps& maps, bool pair, int cluster,
                   int grid, int smem, int most_smem, cudaStream_t stream) {
    const cudaError_t e = raise_smem(once, reinterpret_cast<const void*>(kern), most_smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads_of(pair));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, maps);
}

// Of 227 KiB, less the static arrays.
constexpr int kMostSmem = 227 * 1024 - 1024;

template <bool kF32, bool kPair, bool kTrans, bool kSplit>
cudaError_t launch_rows(const RowsArgs& a, const RowsMaps& maps, int grid, int smem, cudaStream_t stream) {
    static OncePerDevice once;
    return launch(product_rows_kernel<kF32, kPair, kTrans, kSplit>, once, a, maps, kPair, kPair ? 2 : a.split, grid, smem,
                  kMostSmem, stream);
}

int64_t most_tiles(int R, int E, int nt) { return E == 1 ? (R + nt - 1) / nt : mx4_max_tiles(R, E, nt); }

// How rows are multiplied: about twice an expert's average of rows a tile, so
// that most experts are one tile and their weights are read once; from kPairRows
// on by pairs of CTAs.  Units so few that SMs would be idle are split along
// their contraction over a cluster instead: a CTA reads about 100 GB/s, and the
// cluster costs 2 to 4 us, so 40 stages or more, 16 or more a CTA.  16 rows of a
// dense product of 96 stages (6144 -> 4096, 32 units) take 15.6 us by four CTAs a
// unit and 22.5 whole, of 44 stages (2816 -> 2048) 12.0 by two and 12.8, of 32
// stages (2048 -> 6144) 12.1 and 10.6; 256 rows 24 us by two and 33 by pairs.
// (Clusters of eight and four leave some SMs out; `clusters` is how many run at
// once.)
struct How {
    Mx4Tiling t;
    int split;
};
How how_of(int R, int E, int features, int contraction, int sms) {
    const long long want = E == 1 ? R : 2LL * R / E + 16, rows = want < R ? want : R;
    const auto up = [](long long x, int align, int most) {
        return static_cast<int>(x > most ? most : (x + align - 1) / align * align);
    };
    How h{{up(rows, 16, kSingleTileRows), 16}, 1};
    const long long units = most_tiles(R, E, h.t.nt) * ((features + 127) / 128);
    const int stages = (contraction + kBlock - 1) / kBlock;
    for (int split = 2; split <= 8; split *= 2) {
        const int clusters = split == 8 ? sms * 3 / 32 : split == 4 ? sms * 15 / 64 : sms / 2;
        const bool fits = (split - 1) * h.t.nt * 512 <= 96 * 1024;  // the others' sums
        if (units <= clusters && fits && stages >= 40 && stages >= 16 * split) h.split = split;
    }
    if (h.split == 1 && want >= kPairRows && R >= kPairRows) h.t = {up(rows, 32, kPairTileRows), 32};
    return h;
}

// Whether dW's units are 256 x 256, or half of that where twice as many take the
// pairs no more turns: a dense 1000 x 1064 of 4096 rows takes 33.2 us in 20 wide
// units and 27.2 in 36, 256 x 6144 25.6 and 20.1 (24 and 48), of 512 rows in fp32
// 11.4 and 9.6.  With another turn they lose: 2816 x 2048 of 4096 rows 42.3 and
// 43.9 (two and three), 8 experts of 1024 rows, 1000 x 1064, 31.5 and 35.4 (three
// and four); 60 experts of 273 rows, 2816 x 2048, 166 and 239.
bool wide_units(int E, int N, int K, int sms) {
    const auto turns = [&](int wide) {
        const long long units = static_cast<long long>(E) * ((N + 255) / 256) * ((K + wide - 1) / wide);
        return (units + sms / 2 - 1) / (sms / 2);
    };
    return turns(128) > turns(256);
}

}  // namespace

cudaError_t launch_expert_product(const void* x, int64_t ld_x, int R, const void* w, int E, int N, int K, bool trans,
                                  const int32_t* offs, RowsOut y, int* status, int sms, cudaStream_t stream) {
    const How h = how_of(R, E, trans ? K : N, trans ? N : K, sms);
    const Mx4Tiling t = h.t;
    const bool pair = t.align == 32;
    RowsArgs a = {};
    a.plan = {offs, nullptr, E, R, 1, R, t.nt, t.align};
    a.y = y.p;
    a.ld_y = y.ld;
    a.N = trans ? K : N;
    a.C = trans ? N : K;
    a.split = h.split;
    a.status = status;
    RowsMaps maps;
    if (!map3(&maps.w, w, 0, K, N, E, kBlock, trans ? kBlock : 128)) return cudaErrorInvalidValue;
    const int boxes = t.nt / (pair ? 2 : 1) / 16;
    for (int i = 0; i < boxes; ++i)
        if (!map2(&maps.x[i], x, a.C, R, ld_x, pair || 16 * (i + 1) < R ? 16 * (i + 1) : R)) return cudaErrorInvalidValue;
    const int sb = stage_bytes_of(t.nt, pair);
    const int rest = 1024 + (h.split - 1) * t.nt * 512 + epi_bytes(pair) * epi_groups(pair) +
                     plan_ints(E) * static_cast<int>(sizeof(int));
    const int fit = (kMostSmem - rest) / sb;
    a.stages = fit < kMaxStages ? fit : kMaxStages;
    const int smem = a.stages * sb + rest;
    const int split_grid = static_cast<int>(h.split > 1 ? most_tiles(R, E, t.nt) * ((a.N + 127) / 128) * h.split : 0);
    const int grid = pair ? sms / 2 * 2 : h.split > 1 ? split_grid : sms;
    const auto by_way = [&](auto f32, auto two, auto cut) {
        constexpr bool kF = decltype(f32)::value, kP = decltype(two)::value, kS = decltype(cut)::value;
        return trans ? launch_rows<kF, kP, true, kS>(a, maps, grid, smem, stream)
                     : launch_rows<kF, kP, false, kS>(a, maps, grid, smem, stream);
    };
    const auto by_kind = [&](auto f32) {
        using T = std::true_type;
        using F = std::false_type;
        return pair ? by_way(f32, T{}, F{}) : h.split > 1 ? by_way(f32, F{}, T{}) : by_way(f32, F{}, F{});
    };
    return y.f32 ? by_kind(std::true_type{}) : by_kind(std::false_type{});
}

cudaError_t launch_expert_product_grad_w(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, int R, int E, int N,
                                         int K, const int32_t* offs, void* dw, int dw_f32, int* status, int sms,
                                         cudaStream_t stream) {
    WeightsArgs a = {};
    a.plan = {offs, nullptr, E, R, 1, R, kBlock, 16};
    a.N = N;
    a.K = K;
    a.status = status;
    WeightsMaps maps;
    for (int i = 0; i < 7; ++i)
        if (!map2(&maps.dy[i], dy, N, R, ld_dy, kBlock >> i) || !map2(&maps.x[i], x, K, R, ld_x, kBlock >> i))
            return cudaErrorInvalidValue;
    a.whole = N % kBlock == 0 && K % kBlock == 0;
    if (a.whole && (!columns_map(&maps.dy2, dy, N, R, ld_dy) || !columns_map(&maps.x2, x, K, R, ld_x))) return cudaErrorInvalidValue;
    if (!map3(&maps.dw, dw, dw_f32, K, N, E, dw_f32 ? 32 : 64, 32)) return cudaErrorInvalidValue;
    const auto by_width = [&](auto width) {
        constexpr int kWide = decltype(width)::value;
        // six stages of wide units up to 340 experts, five beyond: 64 experts of 384
        // rows (K 6144, N 4096) take 846 us with six and 915 with five
        const int rest = kWEpiBytes + static_cast<int>(sizeof(Shared)) + plan_ints(E) * static_cast<int>(sizeof(int));
        const int fit = (227 * 1024 - rest) / kWStageBytes<kWide>;
        a.stages = fit < kMaxStages ? fit : kMaxStages;
        const int smem = a.stages * kWStageBytes<kWide> + rest;
        static OncePerDevice once[2];
        return dw_f32 ? launch(product_weights_kernel<true, kWide>, once[1], a, maps, true, 2, sms / 2 * 2, smem, 227 * 1024,
                               stream)
                      : launch(product_weights_kernel<false, kWide>, once[0], a, maps, true, 2, sms / 2 * 2, smem,
                               227 * 1024, stream);
    };
    return wide_units(E, N, K, sms) ? by_width(std::integral_constant<int, 256>{})
                                    : by_width(std::integral_constant<int, 128>{});
}

}  // namespace moeq
