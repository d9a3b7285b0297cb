// Operators on any number of tokens around the experts' products: the
// router's top-k and its gradient, the stable sort of (token, slot) pairs by
// expert, and the movement of rows to expert order and back, with gradients.
// All of them move each byte once; what bounds them is HBM (large) or the
// launch (small).
#include <float.h>

#include "moeq_device.cuh"
#include "moeq_rows.h"

namespace moeq {
namespace {

constexpr int kMaxK = MOEQ_MAX_TOPK;

// --------------------------------------------------------------- elements
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Eight consecutive elements, as they sit in memory (raw) and as floats.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int, int) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p, int, int) const { *reinterpret_cast<uint4*>(p) = a; }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        a = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p, int, int) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void store(float* p, int, int) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
};
// Four elements a block's width (`step`) apart, for widths and addresses that
// sixteen bytes at a time do not fit: neighbouring threads still touch
// neighbouring elements, and four loads are in flight (one at a time left a
// 1001-wide fp32 movement at 39 % of the copy rate).  `left`: columns from
// the first on.
template <typename T>
struct RawS {
    T a[4];
    __device__ __forceinline__ void load(const T* p, int left, int step) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * step < left)
                a[i] = p[i * step];
            else
                st1(&a[i], 0.f);
    }
    __device__ __forceinline__ void store(T* p, int left, int step) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * step < left) p[i * step] = a[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) st1(&a[i], 0.f);
    }
    __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(a[i]);
    }
    __device__ __forceinline__ void set(const float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) st1(&a[i], v[i]);
    }
};
template <typename T, int V>
struct RawOf {
    using type = RawS<T>;
};
template <typename T>
struct RawOf<T, 8> {
    using type = Raw8<T>;
};
template <typename T, int V>
using Raw = typename RawOf<T, V>::type;
// A thread's first column in block y of a row.
template <int V>
__device__ __forceinline__ int first_col(int y) {
    return V == 8 ? (y * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8
                  : y * static_cast<int>(blockDim.x) * 4 + static_cast<int>(threadIdx.x);
}

// ------------------------------------------------------------------ router
// A logit as an unsigned key that orders as the logit does; 0 for one that
// is never picked (-inf, NaN).  +inf counts as the largest finite number, so
// that the softmax over the picks stays finite.
__device__ __forceinline__ uint32_t logit_key(float f) {
    if (!(f > -INFINITY)) return 0u;
    const uint32_t u = __float_as_uint(fminf(f, FLT_MAX) + 0.0f);  // -0 folds onto +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float logit_of_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// key[i] = 0 on this lane, for an i that is the same on all: a tree of
// branches, so that keys stay in registers at three branches a call.
template <int N>
__device__ __forceinline__ void clear_key(uint32_t* key, int i, bool me) {
    if constexpr (N == 1) {
        if (me) key[0] = 0u;
    } else {
        if (i < N / 2)
            clear_key<N / 2>(key, i, me);
        else
            clear_key<N / 2>(key + N / 2, i - N / 2, me);
    }
}

// One warp a row: lane l holds the keys of experts l, l + 32, ...; a round
// takes the largest key and the lowest id that holds it (two warp
// reductions), and lane j keeps round j's pick for the softmax.  8191 rows of
// 256 take 8.0 us for eight picks, 5.7 for four and 3.9 for one: the rounds
// bound it, not the 1.3 us of bytes.
template <int NPER>
__global__ void __launch_bounds__(128) route_rows_kernel(const float* logits, int64_t ld, int T, int E,
                                                         int k, int32_t* __restrict__ id, float* __restrict__ w) {
    chain();
    const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= T) return;
    const float* row = logits + t * ld;
    uint32_t key[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < E ? logit_key(row[e]) : 0u;
    }
    int my_id = -1;
    float my_v = 0.f;
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < NPER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (!top) break;  // nothing left that may be picked
        const int e = __reduce_min_sync(0xffffffffu, best == top ? lane + 32 * at : 0x7fffffff);
        clear_key<NPER>(key, e >> 5, (e & 31) == lane);
        if (lane == j) {
            my_id = e;
            my_v = logit_of_key(top);
        }
    }
    const float v0 = __shfl_sync(0xffffffffu, my_v, 0);
    const float p = my_id >= 0 ? expf(my_v - v0) : 0.f;
    float sum = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < k) {
        id[static_cast<int64_t>(t) * k + lane] = my_id;
        w[static_cast<int64_t>(t) * k + lane] = my_id >= 0 ? __fdiv_rn(p, sum) : 0.f;
    }
}

// dl[id_j] = w_j (dw_j - sum_i w_i dw_i), zero elsewhere.  One warp a row:
// zeros first, then the picks (ordered by the warp barrier).  8191 rows of 256:
// 2.7 us.
__global__ void __launch_bounds__(128) route_rows_grad_kernel(const float* dw,
                                                              const int32_t* id,
                                                              const float* w, int T, int E, int k,
                                                              float* __restrict__ dl, int64_t ld, int vec) {
    chain();
    const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= T) return;
    float* row = dl + t * ld;
    float g = 0.f, p = 0.f;
    int e = -1;
    if (lane < k) {
        const int64_t i = static_cast<int64_t>(t) * k + lane;
        e = id[i];
        p = w[i];
        g = dw[i];
    }
    const bool live = e >= 0 && e < E;
    float s = live ? p * g : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (vec) {
        for (int c = lane * 4; c < E; c += 128) *reinterpret_cast<float4*>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
        for (int c = lane; c < E; c += 32) row[c] = 0.f;
    }
    __syncwarp();
    if (live) row[e] = p * (g - s);
}

// -------------------------------------------------------------------- sort
// Stable counting sort of the pairs by expert, with no memory but the outputs.
// A block owns a contiguous chunk of the pairs, and each of its warps a
// contiguous run.
//   1 each warp walks its run 32 pairs at a time, counting experts in bins of
//     its own (shared memory).  Ballots over the bits of the id find the equal
//     ones among the 32 (a match instruction took 1.6 times as long), so a
//     pair's rank in the run is known as it is counted, and scanning the bins
//     over the warps gives its rank in the chunk.  Ranks go to pair_row,
//     the chunk's counts to row_pair;
//   2 every block adds up the counts of the chunks before its own and of all,
//     scans them over the experts, and turns its ranks into rows;
//   3 row_pair is scattered from pair_row (step 2 still reads the counts
//     there).
// One block does all three when it holds every pair.  The steps are chained
// by programmatic launches.  No atomic decides an order, so the result is
// the same every time.  262144 pairs over 256 experts: one cluster of 16
// CTAs that met in distributed shared memory took 19 us, 7 of them in step
// 1's walk on 16 SMs.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortBatch = 2;
// Pairs of a block, at least: with 2048, 262144 pairs over 256 experts take 15.9
// us against 15.7 (step 2 reads twice the counts).
constexpr int kSortChunk = 4096;
// The most blocks: 524288 pairs over 256 experts take 21.1 us with 128, 24.6 with
// 64 (longer runs in step 1).  The most counts (blocks x experts) that step 2
// has every block read: 262144 pairs over 1000 experts take 20.4 us with the 32
// blocks that this leaves and 18.3 with 64, so a higher limit is open; with 256
// experts it does not bind.
constexpr int kSortBlocks = 128, kSortCounts = 32768;
// Pairs that one block sorts alone: 2400 take it 6.2 us, 4096 7.1 and 8000 12.0;
// the three steps take 9.7 us for 4104.
constexpr int kSortOne = 4096;
static_assert(kSortChunk >= 2 * MOEQ_MAX_EXPERTS, "the chunks' counts fit in row_pair");

__device__ __forceinline__ void load_ids(const int32_t* id, int64_t b, int64_t end, int E, int lane,
                                         int (&e)[kSortBatch]) {
#pragma unroll
    for (int i = 0; i < kSortBatch; ++i) {
        const int64_t p = b + i * 32 + lane;
        e[i] = p < end ? id[p] : -1;
    }
#pragma unroll
    for (int i = 0; i < kSortBatch; ++i)
        if (e[i] < 0 || e[i] >= E) e[i] = -1;
}

// The lanes that hold this lane's id (ids of `bits` bits; -1 for none).
__device__ __forceinline__ unsigned same_ids(int e, int bits) {
    unsigned same = __ballot_sync(0xffffffffu, e >= 0);
    for (int i = 0; i < bits; ++i) {
        const unsigned set = __ballot_sync(0xffffffffu, (e >> i) & 1);
        same &= (e >> i) & 1 ? set : ~set;
    }
    return same;
}

// Exclusive scan over the block of one int a thread; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* scratch, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();  // scratch may still be read
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int w = scratch[lane];
    const int own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    return __shfl_sync(0xffffffffu, w - own, warp) + inc - v;
}

struct SortArgs {
    const int32_t* id;
    int P, E, warps, run, bits;
    int32_t *offs, *pair_row, *row_pair;
};

// Step 1; with kOne the block holds every pair and does the rest too.
template <bool kOne>
__global__ void __launch_bounds__(kSortThreads) sort_rank_kernel(const SortArgs a) {
    extern __shared__ int bins[];  // [warps][E], then kOne: [E] first rows
    __shared__ int scratch[kSortWarps];
    chain();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.E;
    const int64_t p0 = (static_cast<int64_t>(blockIdx.x) * a.warps + warp) * a.run;
    const int64_t p1 = warp < a.warps ? min(p0 + a.run, static_cast<int64_t>(a.P)) : p0;
    int* mine = bins + warp * E;
    int e[kSortBatch], ahead[kSortBatch];
    load_ids(a.id, p0, p1, E, lane, e);
    for (int i = tid; i < a.warps * E; i += kSortThreads) bins[i] = 0;
    __syncthreads();
    for (int64_t b = p0; b < p1;) {
        int next[kSortBatch];
        load_ids(a.id, b + kSortBatch * 32, p1, E, lane, next);
#pragma unroll
        for (int i = 0; i < kSortBatch; ++i) {
            const unsigned same = same_ids(e[i], a.bits);
            const int before = __popc(same & ((1u << lane) - 1u));
            const int n = e[i] >= 0 ? mine[e[i]] : 0;
            ahead[i] = n + before;
            __syncwarp();
            if (e[i] >= 0 && before == 0) mine[e[i]] = n + __popc(same);
            __syncwarp();
            const int64_t p = b + i * 32 + lane;
            if (p < p1) a.pair_row[p] = e[i] >= 0 ? ahead[i] : -1;  // the rank in the run, for now
            e[i] = next[i];
        }
        b += kSortBatch * 32;
    }
    __syncthreads();
    int count = 0;
    if (tid < E) {  // one expert a thread: E <= MOEQ_MAX_EXPERTS = kSortThreads
        for (int i = 0; i < a.warps; ++i) {
            const int c = bins[i * E + tid];
            bins[i * E + tid] = count;
            count += c;
        }
        if (!kOne) a.row_pair[static_cast<int64_t>(blockIdx.x) * E + tid] = count;
    }
    int kept = 0;
    int* first = bins + a.warps * E;
    if constexpr (kOne) {
        const int start = block_scan(count, scratch, &kept);
        if (tid < E) {
            first[tid] = start;
            a.offs[tid] = start;
        }
        if (tid == 0) a.offs[E] = kept;
    }
    __syncthreads();
    for (int64_t p = p0 + lane; p < p1; p += 32) {
        const int x = a.id[p];
        if (x < 0 || x >= E) continue;
        const int row = a.pair_row[p] + mine[x] + (kOne ? first[x] : 0);
        a.pair_row[p] = row;
        if (kOne) a.row_pair[row] = static_cast<int32_t>(p);
    }
    if (kOne)
        for (int r = kept + tid; r < a.P; r += kSortThreads) a.row_pair[r] = -1;
}

// Step 2.
__global__ void __launch_bounds__(kSortThreads) sort_rows_kernel(const SortArgs a) {
    __shared__ int before_s[kSortThreads], all_s[kSortThreads], first[MOEQ_MAX_EXPERTS], scratch[kSortWarps];
    chain();
    const int tid = threadIdx.x, E = a.E, blocks = gridDim.x;
    // a power of two of threads for the experts, the rest of the block splits the chunks
    const int log_e = a.bits, e = tid & ((1 << log_e) - 1), sub = tid >> log_e, subs = kSortThreads >> log_e;
    int before = 0, all = 0;
    if (e < E) {
        for (int g0 = sub; g0 < blocks; g0 += 16 * subs) {
            int c[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int g = g0 + i * subs;
                c[i] = g < blocks ? a.row_pair[static_cast<int64_t>(g) * E + e] : 0;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                all += c[i];
                if (g0 + i * subs < static_cast<int>(blockIdx.x)) before += c[i];
            }
        }
    }
    before_s[tid] = before;
    all_s[tid] = all;
    __syncthreads();
    before = all = 0;
    if (tid < E)
        for (int i = 0; i < subs; ++i) {
            before += before_s[(i << log_e) + tid];
            all += all_s[(i << log_e) + tid];
        }
    int kept;
    const int start = block_scan(all, scratch, &kept);
    if (tid < E) {
        first[tid] = start + before;
        if (blockIdx.x == 0) a.offs[tid] = start;
    }
    if (blockIdx.x == 0 && tid == 0) a.offs[E] = kept;
    __syncthreads();
    const int64_t chunk = static_cast<int64_t>(a.warps) * a.run, p0 = blockIdx.x * chunk;
    const int64_t p1 = min(p0 + chunk, static_cast<int64_t>(a.P));
    for (int64_t p = p0 + tid; p < p1; p += kSortThreads) {
        const int x = a.id[p];
        if (x >= 0 && x < E) a.pair_row[p] += first[x];
    }
}

// Step 3.
__global__ void __launch_bounds__(256) sort_pairs_kernel(const SortArgs a) {
    chain();
    const int64_t p = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (p >= a.P) return;
    const int row = a.pair_row[p], kept = a.offs[a.E];
    if (row >= 0) a.row_pair[row] = static_cast<int32_t>(p);
    if (p >= kept) a.row_pair[p] = -1;
}

// ------------------------------------------------------------------ gather
// xs[pair_row[t, j]] = x[t].  Token-major: each of x's elements is read once
// and written to its rows (reading row-major would read it top_k times).
// The rows from offs[E] on are zeroed, shared out over the tokens' blocks.
template <typename T, int V>
__global__ void __launch_bounds__(256) gather_rows_kernel(const T* x, int64_t ld_x, int H, int k,
                                                          const int32_t* offs, int E, int64_t R,
                                                          const int32_t* pair_row, T* __restrict__ xs,
                                                          int64_t ld_xs) {
    chain();
    const int c = first_col<V>(blockIdx.y), left = H - c, step = blockDim.x;
    if (left <= 0) return;
    const int64_t t = blockIdx.x;
    const int kept = max(offs[E], 0);
    Raw<T, V> v;
    v.load(x + t * ld_x + c, left, step);
    const int32_t* pr = pair_row + t * k;
    for (int j0 = 0; j0 < k; j0 += 8) {
        int r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = j0 + j < k ? pr[j0 + j] : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (r[j] >= 0 && r[j] < R) v.store(xs + r[j] * ld_xs + c, left, step);
    }
    v.zero();
    for (int64_t r = kept + t; r < R; r += gridDim.x) v.store(xs + r * ld_xs + c, left, step);
}

// ----------------------------------------------------------------- combine
// out[t] = base[t] + sum_j w[t, j] y[pair_row[t, j]], fp32 in slot order
// (the base first), rounded once.  Each thread holds the loads of up to
// eight rows in flight; slots without a row add nothing.
template <typename TY, typename TO, int V, bool kWeighted>
__global__ void __launch_bounds__(256) combine_rows_kernel(const TY* y, int64_t ld_y, int H, int k,
                                                           int64_t R, const int32_t* pair_row,
                                                           const float* w, const TO* base,
                                                           int64_t ld_base, TO* __restrict__ out, int64_t ld_out) {
    chain();
    const int c = first_col<V>(blockIdx.y), left = H - c, step = blockDim.x;
    if (left <= 0) return;
    const int64_t t = blockIdx.x;
    const int32_t* pr = pair_row + t * k;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    if (base) {
        Raw<TO, V> b;
        b.load(base + t * ld_base + c, left, step);
        b.get(acc);
    }
    for (int j0 = 0; j0 < k; j0 += 8) {
        Raw<TY, V> v[8];
        float ww[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ww[j] = 0.f;
            v[j].zero();
            if (j0 + j < k) {
                const int r = pr[j0 + j];
                if (r >= 0 && r < R) {
                    v[j].load(y + r * ld_y + c, left, step);
                    ww[j] = kWeighted ? w[t * k + j0 + j] : 1.f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float f[V];
            v[j].get(f);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(ww[j], f[i], acc[i]);
        }
    }
    Raw<TO, V> o;
    o.set(acc);
    o.store(out + t * ld_out + c, left, step);
}

// ---------------------------------------------------------- combine's grad
// dy[pair_row[t, j]] = w[t, j] dout[t] and dw[t, j] = <dout[t], y[..]>: one
// block a token, so that dout is read once for all its slots and the dot
// products end in one block reduction (a fixed tree).  The rows of dy from
// offs[E] on are zeroed, shared out over the blocks.
template <typename TY, typename TO, int V, int KM>
__global__ void __launch_bounds__(256) combine_rows_grad_kernel(
    const TO* dout, int64_t ld_do, const TY* y, int64_t ld_y, int H, int k,
    const int32_t* offs, int E, int64_t R, const int32_t* pair_row,
    const float* w, TY* __restrict__ dy, int64_t ld_dy, float* __restrict__ dw) {
    chain();
    const int tid = threadIdx.x, step = blockDim.x;
    const int kept = max(offs[E], 0);
    __shared__ float red[8][KM];
    const int64_t t = blockIdx.x;
    int row[KM];
    float ww[KM], dot[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        row[j] = -1;
        ww[j] = dot[j] = 0.f;
        if (j < k) {
            const int r = pair_row[t * k + j];
            if (r >= 0 && r < R) {
                row[j] = r;
                ww[j] = w[t * k + j];
            }
        }
    }
    for (int c = first_col<V>(0); c < H; c += step * V) {
        Raw<TO, V> d;
        d.load(dout + t * ld_do + c, H - c, step);
        float df[V];
        d.get(df);
        // rows in flight at a time: eight 16-byte loads, or four of RawS's
        // (which would need twice the registers)
        constexpr int kGroup = V == 8 && KM >= 8 ? 8 : 4;
#pragma unroll
        for (int j0 = 0; j0 < KM; j0 += kGroup) {
            if (j0 >= k) break;
            Raw<TY, V> v[kGroup];
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                v[j].zero();
                if (row[j0 + j] >= 0) v[j].load(y + row[j0 + j] * ld_y + c, H - c, step);
            }
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                if (row[j0 + j] < 0) continue;
                float f[V], g[V];
                v[j].get(f);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dot[j0 + j] = fmaf(df[i], f[i], dot[j0 + j]);
                    g[i] = ww[j0 + j] * df[i];
                }
                Raw<TY, V> o;
                o.set(g);
                o.store(dy + row[j0 + j] * ld_dy + c, H - c, step);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        float s = dot[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if ((tid & 31) == 0) red[tid >> 5][j] = s;
    }
    __syncthreads();
    if (tid < k) {
        float s = 0.f;
        for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += red[i][tid];
        dw[t * k + tid] = s;
    }
    Raw<TY, V> z;
    z.zero();
    for (int64_t r = kept + t; r < R; r += gridDim.x)
        for (int c = first_col<V>(0); c < H; c += step * V) z.store(dy + r * ld_dy + c, H - c, step);
}

// Eight elements at a time fit when rows start and step on 16 bytes.
bool fits8(const void* p, int64_t ld, int f32) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (f32 ? 4 : 8) == 0;
}

template <typename F>
cudaError_t by_type(int f32, F f) {
    return f32 ? f(static_cast<float*>(nullptr)) : f(static_cast<__nv_bfloat16*>(nullptr));
}

}  // namespace

cudaError_t raise_smem(OncePerDevice& once, const void* kernel, int bytes) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return once.on(dev, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
}

cudaError_t launch_route_rows(const float* logits, int64_t ld, int T, int E, int k, int32_t* id, float* w,
                              cudaStream_t stream) {
    const auto kern = E <= 64 ? route_rows_kernel<2> : E <= 256 ? route_rows_kernel<8> : route_rows_kernel<32>;
    return launch_chained(kern, (T + 3) / 4, 128, 0, stream, logits, ld, T, E, k, id, w);
}

cudaError_t launch_route_rows_grad(const float* dw, const int32_t* id, const float* w, int T, int E, int k,
                                   float* dlogits, int64_t ld, cudaStream_t stream) {
    const int vec = E % 4 == 0 && fits8(dlogits, ld, 1);
    return launch_chained(route_rows_grad_kernel, (T + 3) / 4, 128, 0, stream, dw, id, w, T, E, k, dlogits, ld, vec);
}

cudaError_t launch_expert_sort(const int32_t* id, int T, int k, int E, int32_t* offs, int32_t* pair_row,
                               int32_t* row_pair, cudaStream_t stream) {
    SortArgs a = {id, T * k, E, 0, 0, 0, offs, pair_row, row_pair};
    // one block for few pairs; else chunks of kSortChunk, longer ones beyond the most blocks
    const int most = min(kSortBlocks, kSortCounts / E);
    const int blocks = a.P <= kSortOne ? 1 : min(most, (a.P + kSortChunk - 1) / kSortChunk);
    const int chunk = (a.P + blocks - 1) / blocks;
    a.warps = min(kSortWarps, max(1, (chunk + 31) / 32));
    a.run = (chunk + a.warps - 1) / a.warps;
    while ((1 << a.bits) < E) ++a.bits;
    const auto rank = blocks == 1 ? sort_rank_kernel<true> : sort_rank_kernel<false>;
    static OncePerDevice once[2];
    cudaError_t e = raise_smem(once[blocks == 1], reinterpret_cast<const void*>(rank),
                               (kSortWarps + 1) * MOEQ_MAX_EXPERTS * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
    e = launch_chained(rank, blocks, kSortThreads, (a.warps + 1) * E * sizeof(int), stream, a);
    if (e != cudaSuccess || blocks == 1) return e;
    e = launch_chained(sort_rows_kernel, blocks, kSortThreads, 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_chained(sort_pairs_kernel, (a.P + 255) / 256, 256, 0, stream, a);
}

cudaError_t launch_gather_rows(RowsIn x, int T, int H, int k, const int32_t* offs, int E, const int32_t* pair_row,
                               RowsOut xs, cudaStream_t stream) {
    const bool v8 = H % 8 == 0 && fits8(x.p, x.ld, x.f32) && fits8(xs.p, xs.ld, x.f32);
    return by_type(x.f32, [&](auto* tag) {
        using Ty = std::remove_pointer_t<decltype(tag)>;
        const int nv = v8 ? H / 8 : (H + 3) / 4, threads = nv >= 256 ? 256 : (nv + 31) / 32 * 32;
        const dim3 grid(T, (nv + threads - 1) / threads);
        const Ty* xp = static_cast<const Ty*>(x.p);
        Ty* sp = static_cast<Ty*>(xs.p);
        return launch_chained(v8 ? gather_rows_kernel<Ty, 8> : gather_rows_kernel<Ty, 4>, grid, threads, 0, stream, xp, x.ld,
                              H, k, offs, E, static_cast<int64_t>(T) * k, pair_row, sp, xs.ld);
    });
}

cudaError_t launch_combine_rows(RowsIn y, int T, int H, int k, const int32_t* pair_row, const float* w, RowsIn base,
                                RowsOut out, cudaStream_t stream) {
    const bool v8 = H % 8 == 0 && fits8(y.p, y.ld, y.f32) && fits8(out.p, out.ld, out.f32) &&
                    (!base.p || fits8(base.p, base.ld, out.f32));
    const int64_t R = static_cast<int64_t>(T) * k;
    return by_type(y.f32, [&](auto* ty) {
        return by_type(out.f32, [&](auto* to) {
            using TY = std::remove_pointer_t<decltype(ty)>;
            using TO = std::remove_pointer_t<decltype(to)>;
            const int nv = v8 ? H / 8 : (H + 3) / 4, threads = nv >= 256 ? 256 : (nv + 31) / 32 * 32;
            const dim3 grid(T, (nv + threads - 1) / threads);
            const TY* yp = static_cast<const TY*>(y.p);
            const TO* bp = static_cast<const TO*>(base.p);
            TO* op = static_cast<TO*>(out.p);
            auto go = [&](auto kern) {
                return launch_chained(kern, grid, threads, 0, stream, yp, y.ld, H, k, R, pair_row, w, bp, base.ld, op, out.ld);
            };
            if (v8) return w ? go(combine_rows_kernel<TY, TO, 8, true>) : go(combine_rows_kernel<TY, TO, 8, false>);
            return w ? go(combine_rows_kernel<TY, TO, 4, true>) : go(combine_rows_kernel<TY, TO, 4, false>);
        });
    });
}

cudaError_t launch_combine_rows_grad(RowsIn dout, RowsIn y, int T, int H, int k, const int32_t* offs, int E,
                                     const int32_t* pair_row, const float* w, RowsOut dy, float* dw,
                                     cudaStream_t stream) {
    const bool v8 = H % 8 == 0 && fits8(y.p, y.ld, y.f32) && fits8(dout.p, dout.ld, dout.f32) &&
                    fits8(dy.p, dy.ld, y.f32);
    const int64_t R = static_cast<int64_t>(T) * k;
    return by_type(y.f32, [&](auto* ty) {
        return by_type(dout.f32, [&](auto* to) {
            using TY = std::remove_pointer_t<decltype(ty)>;
            using TO = std::remove_pointer_t<decltype(to)>;
            const int grid = T;
            auto go = [&](auto kern) {
                return launch_chained(kern, grid, 256, 0, stream, static_cast<const TO*>(dout.p), dout.ld,
                                      static_cast<const TY*>(y.p), y.ld, H, k, offs, E, R, pair_row, w,
                                      static_cast<TY*>(dy.p), dy.ld, dw);
            };
            if (k <= 4)
                return v8 ? go(combine_rows_grad_kernel<TY, TO, 8, 4>) : go(combine_rows_grad_kernel<TY, TO, 4, 4>);
            if (k <= 8)
                return v8 ? go(combine_rows_grad_kernel<TY, TO, 8, 8>) : go(combine_rows_grad_kernel<TY, TO, 4, 8>);
            return v8 ? go(combine_rows_grad_kernel<TY, TO, 8, kMaxK>) : go(combine_rows_grad_kernel<TY, TO, 4, kMaxK>);
        });
    });
}

}  // namespace moeq
