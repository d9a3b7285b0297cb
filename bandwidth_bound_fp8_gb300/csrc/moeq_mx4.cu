// MXFP4 (OCP microscaling) quantisation: blocks of 32 along K share the scale
// 2^s, s = max(floor(log2 amax) - 2, -127), stored as the byte s + 127; an
// element is the E2M1 code of x * 2^-s, rounded to nearest even, saturating
// at 6.  x * 2^-s is exact (a power of two; where it underflows the code is 0
// either way), so codes and scales are the definition's bit for bit.  A block
// that holds a NaN or an infinity gets the scale 255, E8M0's NaN.
#include "moeq_device.cuh"
#include "moeq_mx4_plan.cuh"
#include "moeq_rows.h"

namespace moeq {
namespace {

constexpr uint32_t kNanScale = 255;

__device__ __forceinline__ float pow2_bits(int biased) { return __uint_as_float(static_cast<uint32_t>(biased) << 23); }

// Scale byte of a block from its largest magnitude (as bits, so that a NaN
// compares above everything).
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return kNanScale;
    // subnormal magnitudes lie below 2^-126: s clamps to -127 for all of them
    const int e = static_cast<int>(amax_bits >> 23) - 2;  // biased exponent of 2^s
    return e > 0 ? static_cast<uint32_t>(e) : 0u;
}

// 2^-s for the scale byte b = s + 127 in [0, 252]: biased exponent 254 - b.
__device__ __forceinline__ float mx4_inverse(uint32_t b) { return pow2_bits(254 - static_cast<int>(b)); }

// Eight floats, scaled, to eight codes (element i in bits 4i..).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], float inv) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(v[0] * inv), "f"(v[1] * inv), "f"(v[2] * inv), "f"(v[3] * inv), "f"(v[4] * inv), "f"(v[5] * inv),
          "f"(v[6] * inv), "f"(v[7] * inv));
    return r;
}

// Four lanes hold a block of 32: the largest of their magnitudes (as fp32
// bits).
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// The block's scale byte (the same in its four lanes) and this lane's codes.
__device__ __forceinline__ uint32_t mx4_block(const float (&v)[8], uint32_t amax, uint32_t* scale) {
    const uint32_t b = mx4_scale_byte(amax);
    *scale = b;
    return b == kNanScale ? 0u : e2m1x8(v, mx4_inverse(b));
}

// Eight consecutive elements as they sit in memory: loaded early, converted
// when they are used.
template <bool kF32>
struct Raw8 {
    uint4 a, b;  // b: fp32 alone
    template <bool kVec>
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if constexpr (kVec) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (kF32 ? 4 : 2));
            a = q[0];
            if constexpr (kF32) b = q[1];
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < (kF32 ? 8 : 4); ++i) {
                if constexpr (kF32) {
                    w[i] = static_cast<const uint32_t*>(p)[at + i];
                } else {
                    const uint16_t* h = static_cast<const uint16_t*>(p) + at + 2 * i;
                    w[i] = h[0] | static_cast<uint32_t>(h[1]) << 16;
                }
            }
            a = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (kF32) b = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    // The largest magnitude, as fp32 bits: bf16 two at a time.
    __device__ __forceinline__ uint32_t amax() const {
        constexpr uint32_t kAbs = kF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
        if constexpr (kF32) {
            return max(max(max(a.x & kAbs, a.y & kAbs), max(a.z & kAbs, a.w & kAbs)),
                       max(max(b.x & kAbs, b.y & kAbs), max(b.z & kAbs, b.w & kAbs)));
        } else {
            const uint32_t m = __vmaxu2(__vmaxu2(a.x & kAbs, a.y & kAbs), __vmaxu2(a.z & kAbs, a.w & kAbs));
            return max(m & 0xFFFF0000u, m << 16);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < (kF32 ? 8 : 4); ++i) {
            if constexpr (kF32) {
                v[i] = __uint_as_float(u[i]);
            } else {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            }
        }
    }
};

// silu(g) * u.  The fast exponential and division are within a few ulp times
// |g|, far below the 4-bit rounding that follows.
__device__ __forceinline__ float swiglu(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

// A warp's segment of a row: kBlocks K blocks of 256 columns, eight of each a
// lane (its loads all issued before the first is used): 2 KiB a warp.
constexpr int kSegment = 4;
__host__ __device__ constexpr int segment_blocks(bool f32, bool swiglu) {
    const int n = kSegment / (f32 ? 2 : 1) / (swiglu ? 2 : 1);
    return n > 0 ? n : 1;
}
__host__ __device__ constexpr int segments(int K, int blocks) { return (mx4_kb(K) + blocks - 1) / blocks; }

template <bool kF32, bool kVec, bool kSwiglu>
struct Segment {
    static constexpr int kBlocks = segment_blocks(kF32, kSwiglu);
    Raw8<kF32> v[kBlocks], u[kSwiglu ? kBlocks : 1];
    __device__ __forceinline__ void load(const void* x, int64_t row0, int seg, int lane, int K) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            const int c = (seg * kBlocks + i) * kMx4TileCols + lane * 8;
            v[i].zero();
            if constexpr (kSwiglu) u[i].zero();
            if (c < K) {
                v[i].template load<kVec>(x, row0 + c);
                if constexpr (kSwiglu) u[i].template load<kVec>(x, row0 + K + c);
            }
        }
    }
    // Codes and scale byte of K block i; a column past K gives zeros.
    __device__ __forceinline__ uint32_t quant(int i, bool in, uint32_t* s) const {
        float f[8];
        v[i].get(f);
        uint32_t m = 0;
        if constexpr (kSwiglu) {
            float g[8];
            u[i].get(g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[j] = swiglu(f[j], g[j]);
                m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
            }
        } else {
            m = v[i].amax();
        }
        const uint32_t q = mx4_block(f, block_max(m), s);
        if (!in) *s = 0;
        return in ? q : 0u;
    }
};

// Rows of activations: resident warps take a segment at a time, the next one's
// loads in flight while this one is quantised.
template <bool kF32, bool kVec, bool kSwiglu>
__global__ void __launch_bounds__(256) quant_act_kernel(const void* x, int64_t ld, int rows, int K,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    chain();
    using Seg = Segment<kF32, kVec, kSwiglu>;
    constexpr int kBlocks = Seg::kBlocks;
    const int lane = threadIdx.x & 31, segs = segments(K, kBlocks), pitch = mx4_scale_pitch(K);
    const unsigned step = gridDim.x * 8, step_rows = step / segs, step_segs = step % segs;
    const unsigned it = blockIdx.x * 8 + (threadIdx.x >> 5);
    int64_t row = it / segs;
    int seg = it % segs;
    if (row >= rows) return;
    Seg g, next;
    g.load(x, row * ld, seg, lane, K);
    for (;;) {
        int64_t next_row = row + step_rows;
        int next_seg = seg + step_segs;
        if (next_seg >= segs) {
            next_seg -= segs;
            ++next_row;
        }
        const bool more = next_row < rows;
        if (more) next.load(x, next_row * ld, next_seg, lane, K);
        uint8_t* q_at = codes + row * (K >> 1) + seg * (kBlocks * kMx4TileCols / 2) + lane * 4;
        uint8_t* s_at = scales + row * pitch + seg * (kBlocks * 8) + (lane >> 2);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            const int kb = seg * kBlocks + i, c = kb * kMx4TileCols + lane * 8;
            if (kb * kMx4TileCols >= K) break;
            uint32_t s;
            const uint32_t q = g.quant(i, c < K, &s);
            if (c < K) *reinterpret_cast<uint32_t*>(q_at + i * (kMx4TileCols / 2)) = q;
            if ((lane & 3) == 0) s_at[i * 8] = static_cast<uint8_t>(s);
        }
        if (!more) return;
        g = next;
        row = next_row;
        seg = next_seg;
    }
}

// Codes and scales back to values.  A value is a code (at most two
// significant bits) times a power of two: exact in bf16 and in fp32 (a
// subnormal of at least 2^-128 fits both; past 2^128 it is an infinity).  The
// scale is applied in two halves, because 2^-127 is no normal number.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) dequant_act_kernel(const uint8_t* codes, const uint8_t* scales, int rows, int K,
                                                          T* __restrict__ out, int64_t ld) {
    chain();
    const int lane = threadIdx.x & 31, segs = segments(K, kSegment);
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t row = item / segs;
    const int seg = static_cast<int>(item - row * segs);
    if (row >= rows) return;
    uint32_t q[kSegment], sc[kSegment];
#pragma unroll
    for (int i = 0; i < kSegment; ++i) {
        const int c = (seg * kSegment + i) * kMx4TileCols + lane * 8;
        q[i] = sc[i] = 0;
        if (c < K) {
            q[i] = *reinterpret_cast<const uint32_t*>(codes + row * (K >> 1) + (c >> 1));
            sc[i] = scales[row * mx4_scale_pitch(K) + (c >> 5)];
        }
    }
#pragma unroll
    for (int i = 0; i < kSegment; ++i) {
        const int c = (seg * kSegment + i) * kMx4TileCols + lane * 8;
        if (c >= K) break;
        const int half = (static_cast<int>(sc[i]) - 127) >> 1, rest = static_cast<int>(sc[i]) - 127 - half;
        const float f0 = pow2_bits(half + 127), f1 = pow2_bits(rest + 127);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h;  // two codes to two exact halves
            asm("{\n .reg .b8 b;\n cvt.u8.u32 b, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}" : "=r"(h) : "r"((q[i] >> (8 * j)) & 0xFFu));
            const float2 f = f16x2_to_f32x2(h);
            v[2 * j] = f.x * f0 * f1;
            v[2 * j + 1] = f.y * f0 * f1;
        }
        if (sc[i] == kNanScale)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(0x7FFFFFFFu);
        T* o = out + row * ld + c;
        if constexpr (sizeof(T) == 4) {
            if constexpr (kVec) {
                reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = v[j];
            }
        } else if constexpr (kVec) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                u[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __float2bfloat16_rn(v[j]);
        }
    }
}

// Where a lane's eight elements of (row r, its 32 lanes = 256 columns) go in
// a weight tile, and its block's scale byte.
__device__ __forceinline__ void store_tile(uint8_t* tile, uint8_t* stile, int r, int lane, uint32_t q, uint32_t s) {
    const int chunk = lane >> 2;
    *reinterpret_cast<uint32_t*>(tile + r * 128 + ((chunk ^ (r & 7)) << 4) + (lane & 3) * 4) = q;
    if ((lane & 3) == 0)
        stile[(lane >> 4) * 512 + (r & 31) * 16 + (r >> 5) * 4 + ((lane >> 2) & 3)] = static_cast<uint8_t>(s);
}

// One block of eight warps a tile, one row a warp at a time.
template <bool kF32, bool kVec>
__global__ void __launch_bounds__(256) quant_weight_kernel(const void* __restrict__ w, int N, int K,
                                                           uint8_t* __restrict__ tiles, uint8_t* __restrict__ stiles) {
    const int kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z, lane = threadIdx.x & 31;
    const int64_t t = (static_cast<int64_t>(e) * gridDim.y + nb) * gridDim.x + kb;
    const int c = kb * kMx4TileCols + lane * 8;
#pragma unroll 4
    for (int r = threadIdx.x >> 5; r < kMx4TileRows; r += 8) {
        const int n = nb * kMx4TileRows + r;
        Raw8<kF32> raw;
        raw.zero();
        const bool in = n < N && c < K;
        if (in) raw.template load<kVec>(w, (static_cast<int64_t>(e) * N + n) * K + c);
        float v[8];
        raw.get(v);
        uint32_t s;
        const uint32_t q = mx4_block(v, block_max(raw.amax()), &s);
        store_tile(tiles + t * kMx4TileBytes, stiles + t * kMx4TileScaleBytes, r, lane, in ? q : 0u, in ? s : 0u);
    }
}

__global__ void __launch_bounds__(256) pack_weight_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, int N, int K,
                                                          uint8_t* __restrict__ tiles, uint8_t* __restrict__ stiles) {
    const int kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z, lane = threadIdx.x & 31;
    const int64_t t = (static_cast<int64_t>(e) * gridDim.y + nb) * gridDim.x + kb;
    const int c = kb * kMx4TileCols + lane * 8;
#pragma unroll 4
    for (int r = threadIdx.x >> 5; r < kMx4TileRows; r += 8) {
        const int n = nb * kMx4TileRows + r;
        const int64_t row = static_cast<int64_t>(e) * N + n;
        uint32_t q = 0, s = 0;
        if (n < N && c < K) {
            q = __ldg(reinterpret_cast<const uint32_t*>(codes + row * (K >> 1) + (c >> 1)));
            s = __ldg(scales + row * (K >> 5) + (c >> 5));
        }
        store_tile(tiles + t * kMx4TileBytes, stiles + t * kMx4TileScaleBytes, r, lane, q, s);
    }
}

// The token tiles of a product: rows gathered into expert order, quantised on
// the way (or copied from codes), and laid out as the tensor core reads them,
// so that the product fetches a stage with plain bulk copies.  The columns
// past K of a row's last block of 256 are zeroed (padding rows of a tile are
// not: they only reach rows of the product that are not stored).
struct Place {
    int64_t block0;  // the row's tile's first K block
    int pos;         // the row's place in its tile
};
__device__ __forceinline__ Place place_of(const PlanShared& plan, const Mx4Plan& p, int r, int kb_all) {
    const int e = plan_find(plan.first, p.E, r);
    const int per = plan_rows_per_tile(plan.first[e + 1] - plan.first[e], p.nt, p.align);
    const int in_e = r - plan.first[e], t = in_e / per;
    return {static_cast<int64_t>(plan.tile[e] + t) * kb_all, in_e - t * per};
}
// Byte offset, inside a K block's scales, of the word of row `pos` and the
// block's 128-column half `kc`.
__device__ __forceinline__ int scale_at(int pos, int kc, int sb) {
    return kc * (sb >> 1) + (pos >> 7) * 512 + (pos & 31) * 16 + ((pos >> 5) & 3) * 4;
}
__device__ __forceinline__ int act_row(const Mx4Plan& p, int r) {
    return min(p.row_pair ? max(p.row_pair[r], 0) / p.top_k : r, p.rows - 1);
}

// From rows to quantise: a warp takes every `parts`-th segment of a row at a
// time (parts = 1 where there are rows for all warps), and finds the row's
// place once.  The next segment's loads are in flight while one is
// quantised; the first one's need only the row number, not the plan.
template <bool kF32, bool kVec, bool kSwiglu>
__global__ void __launch_bounds__(kPlanThreads) act_tiles_kernel(RowsIn x, Mx4Plan p, int K, int parts,
                                                                 uint8_t* __restrict__ tiles,
                                                                 uint8_t* __restrict__ stiles) {
    chain();
    __shared__ int plan_mem[plan_ints(MOEQ_MAX_EXPERTS)];
    const PlanShared plan = plan_at(plan_mem, p.E);
    using Seg = Segment<kF32, kVec, kSwiglu>;
    constexpr int kBlocks = Seg::kBlocks;
    const int lane = threadIdx.x & 31, kb_all = mx4_kb(K), segs = segments(K, kBlocks), sb = mx4_tile_scale_bytes(p.nt);
    const unsigned it = blockIdx.x * (kPlanThreads / 32) + (threadIdx.x >> 5);
    const int step = gridDim.x * (kPlanThreads / 32) / parts, part = it % parts;
    int64_t r = it / parts;  // parts divides the grid's warps, so r steps evenly
    int seg = part;
    Seg g, next;
    int next_row = 0;  // the activation row after this one
    if (r < p.R) {
        g.load(x.p, act_row(p, static_cast<int>(r)) * x.ld, seg, lane, K);
        if (r + step < p.R) next_row = act_row(p, static_cast<int>(r + step));
    }
    int64_t row = r < p.R ? act_row(p, static_cast<int>(r)) : 0;
    plan_scan(p, plan);
    const int r0 = plan.first[0], r1 = plan.first[p.E];
    while (r < r1) {
        const Place at = place_of(plan, p, max(static_cast<int>(r), r0), kb_all);
        const int c_at = at.pos * 128 + (((lane >> 2) ^ (at.pos & 7)) << 4) + (lane & 3) * 4;
        const int s_at = scale_at(at.pos, lane >> 4, sb) + ((lane >> 2) & 3);
        const bool keep = r >= r0;
        for (; seg < segs; seg += parts) {
            // the next segment, of this row or the next
            if (seg + parts < segs)
                next.load(x.p, row * x.ld, seg + parts, lane, K);
            else if (r + step < r1)
                next.load(x.p, static_cast<int64_t>(next_row) * x.ld, part, lane, K);
            uint8_t* t_at = tiles + (at.block0 + seg * kBlocks) * p.nt * 128 + c_at;
            uint8_t* st_at = stiles + (at.block0 + seg * kBlocks) * sb + s_at;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                const int kb = seg * kBlocks + i;
                if (kb >= kb_all) break;
                uint32_t s;
                const uint32_t q = g.quant(i, kb * kMx4TileCols + lane * 8 < K, &s);
                if (!keep) continue;
                *reinterpret_cast<uint32_t*>(t_at + i * (p.nt * 128)) = q;
                if ((lane & 3) == 0) st_at[i * sb] = static_cast<uint8_t>(s);
            }
            g = next;
        }
        seg = part;
        row = next_row;
        r += step;
        if (r + step < r1) next_row = act_row(p, static_cast<int>(r + step));
    }
}

// From codes: a warp moves a row, 16 bytes a lane at a time, up to 8192
// columns' loads in flight.  Scales go a tile a block, a row a thread in the
// order of the tile's words, so that a warp writes 128 bytes in one piece
// (row by row, a third of the kernel's 57 us for 65536 rows of 6144 went into
// their scattered words).
__global__ void __launch_bounds__(kPlanThreads) code_tiles_kernel(const uint8_t* codes, const uint8_t* scales, Mx4Plan p,
                                                                  int K,
                                                                  uint8_t* __restrict__ tiles,
                                                                  uint8_t* __restrict__ stiles) {
    chain();
    __shared__ int plan_mem[plan_ints(MOEQ_MAX_EXPERTS)];
    const PlanShared plan = plan_at(plan_mem, p.E);
    plan_scan(p, plan);
    constexpr int kWide = 8;
    const int lane = threadIdx.x & 31, kb_all = mx4_kb(K), sb = mx4_tile_scale_bytes(p.nt), pitch = mx4_scale_pitch(K);
    const int chunks = K >> 5, all_chunks = kb_all * 8, r0 = plan.first[0], r1 = plan.first[p.E];
    const int step = gridDim.x * (kPlanThreads / 32);
    int64_t r = r0 + blockIdx.x * (kPlanThreads / 32) + (threadIdx.x >> 5);
    int64_t row = r < r1 ? act_row(p, static_cast<int>(r)) : 0;
    while (r < r1) {
        const int64_t next_row = r + step < r1 ? act_row(p, static_cast<int>(r + step)) : 0;
        const uint4* src = reinterpret_cast<const uint4*>(codes + row * (K >> 1));
        const Place at = place_of(plan, p, static_cast<int>(r), kb_all);
        uint8_t* t_at = tiles + (at.block0 * p.nt + at.pos) * 128;
        for (int c0 = 0; c0 < all_chunks; c0 += kWide * 32) {
            uint4 v[kWide];
#pragma unroll
            for (int i = 0; i < kWide; ++i) {
                const int c = c0 + i * 32 + lane;
                v[i] = c < chunks ? src[c] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kWide; ++i) {
                const int c = c0 + i * 32 + lane;
                if (c < all_chunks)
                    *reinterpret_cast<uint4*>(t_at + static_cast<int64_t>(c >> 3) * (p.nt * 128) +
                                              (((c & 7) ^ (at.pos & 7)) << 4)) = v[i];
            }
        }
        r += step;
        row = next_row;
    }
    const int pos = (threadIdx.x & 128) + ((threadIdx.x & 127) >> 2) + (threadIdx.x & 3) * 32;
    for (int g = blockIdx.x; g < plan.tile[p.E]; g += gridDim.x) {
        const int e = plan_find(plan.tile, p.E, g), cnt = plan.first[e + 1] - plan.first[e];
        const int per = plan_rows_per_tile(cnt, p.nt, p.align), i = (g - plan.tile[e]) * per + pos;
        if (pos >= per || i >= cnt) continue;
        const uint2* from = reinterpret_cast<const uint2*>(scales + static_cast<int64_t>(act_row(p, plan.first[e] + i)) * pitch);
        uint8_t* to = stiles + static_cast<int64_t>(g) * kb_all * sb + scale_at(pos, 0, sb);
#pragma unroll 8
        for (int kb = 0; kb < kb_all; ++kb) {
            const uint2 w = from[kb];
            *reinterpret_cast<uint32_t*>(to + static_cast<int64_t>(kb) * sb) = w.x;
            *reinterpret_cast<uint32_t*>(to + static_cast<int64_t>(kb) * sb + (sb >> 1)) = w.y;
        }
    }
}

// The product's CTAs start while the tiles are filled, so an SM that fills
// them keeps its shared memory as the product wants it (an SM changes the
// split with L1 only when it is empty: 48 of 152 CTAs started 2 us late).  A
// preference: a failure costs time, not the product.
template <typename K>
void beside_product(OncePerDevice& once, K kernel) {
    int dev = 0;
    const auto set = [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    };
    if (cudaGetDevice(&dev) != cudaSuccess || once.on(dev, set) != cudaSuccess) cudaGetLastError();
}

bool fits(const void* p, int64_t ld, int f32) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (f32 ? 4 : 8) == 0;
}

}  // namespace

cudaError_t launch_mx4_quant_act(RowsIn x, int rows, int K, int act, uint8_t* codes, uint8_t* scales,
                                 int sms, cudaStream_t stream) {
    const int64_t want = (static_cast<int64_t>(rows) * segments(K, segment_blocks(x.f32, act)) + 7) / 8;
    const unsigned grid = static_cast<unsigned>(want < sms * 4 ? want : sms * 4);
    // the second half of a SwiGLU row starts K elements on: K is a multiple of 32
    const bool vec = fits(x.p, x.ld, x.f32);
    auto go = [&](auto kern) { return launch_chained(kern, grid, 256, 0, stream, x.p, x.ld, rows, K, codes, scales); };
    if (x.f32) {
        if (act) return vec ? go(quant_act_kernel<true, true, true>) : go(quant_act_kernel<true, false, true>);
        return vec ? go(quant_act_kernel<true, true, false>) : go(quant_act_kernel<true, false, false>);
    }
    if (act) return vec ? go(quant_act_kernel<false, true, true>) : go(quant_act_kernel<false, false, true>);
    return vec ? go(quant_act_kernel<false, true, false>) : go(quant_act_kernel<false, false, false>);
}

cudaError_t launch_mx4_dequant_act(const uint8_t* codes, const uint8_t* scales, int rows, int K, RowsOut out,
                                   cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(rows) * segments(K, kSegment) + 7) / 8);
    const bool vec = fits(out.p, out.ld, out.f32);
    auto go = [&](auto* o, auto kern) {
        return launch_chained(kern, grid, 256, 0, stream, codes, scales, rows, K, o, out.ld);
    };
    if (out.f32) {
        float* o = static_cast<float*>(out.p);
        return vec ? go(o, dequant_act_kernel<float, true>) : go(o, dequant_act_kernel<float, false>);
    }
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out.p);
    return vec ? go(o, dequant_act_kernel<__nv_bfloat16, true>) : go(o, dequant_act_kernel<__nv_bfloat16, false>);
}

cudaError_t launch_mx4_quant_weight(const void* w, int w_f32, int E, int N, int K, uint8_t* tiles, uint8_t* stiles,
                                    cudaStream_t stream) {
    const dim3 grid(mx4_kb(K), mx4_nb(N), E);
    const bool vec = fits(w, K, w_f32);
    auto go = [&](auto kern) {
        kern<<<grid, 256, 0, stream>>>(w, N, K, tiles, stiles);
        return cudaGetLastError();
    };
    if (w_f32) return vec ? go(quant_weight_kernel<true, true>) : go(quant_weight_kernel<true, false>);
    return vec ? go(quant_weight_kernel<false, true>) : go(quant_weight_kernel<false, false>);
}

cudaError_t launch_mx4_pack_weight(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, uint8_t* tiles,
                                   uint8_t* stiles, cudaStream_t stream) {
    const dim3 grid(mx4_kb(K), mx4_nb(N), E);
    pack_weight_kernel<<<grid, 256, 0, stream>>>(codes, scales, N, K, tiles, stiles);
    return cudaGetLastError();
}

cudaError_t launch_mx4_act_tiles(const Mx4Source& src, const Mx4Plan& plan, int K, uint8_t* tiles, uint8_t* stiles,
                                 int sms, cudaStream_t stream) {
    // one wave of resident blocks: each scans the plan once
    const int most = sms * 4;
    if (src.codes) {
        const int blocks = (plan.R + 7) / 8;
        static OncePerDevice once;
        beside_product(once, code_tiles_kernel);
        return launch_chained(code_tiles_kernel, blocks < most ? blocks : most, kPlanThreads, 0, stream, src.codes,
                              src.scales, plan, K, tiles, stiles);
    }
    // a warp a row where that fills the wave, else up to eight (a power of two: it divides a block's warps)
    const int segs = segments(K, segment_blocks(src.x.f32, src.act));
    int parts = 1;
    while (parts < 8 && parts < segs && static_cast<int64_t>(plan.R) * parts < most * 8) parts *= 2;
    const int64_t want = (static_cast<int64_t>(plan.R) * parts + 7) / 8;
    const unsigned grid = static_cast<unsigned>(want < most ? want : most);
    const bool vec = fits(src.x.p, src.x.ld, src.x.f32);
    static OncePerDevice once[2][2][2];
    auto go = [&](auto kern) {
        beside_product(once[src.x.f32 != 0][vec][src.act != 0], kern);
        return launch_chained(kern, grid, kPlanThreads, 0, stream, src.x, plan, K, parts, tiles, stiles);
    };
    if (src.x.f32) {
        if (src.act) return vec ? go(act_tiles_kernel<true, true, true>) : go(act_tiles_kernel<true, false, true>);
        return vec ? go(act_tiles_kernel<true, true, false>) : go(act_tiles_kernel<true, false, false>);
    }
    if (src.act) return vec ? go(act_tiles_kernel<false, true, true>) : go(act_tiles_kernel<false, false, true>);
    return vec ? go(act_tiles_kernel<false, true, false>) : go(act_tiles_kernel<false, false, false>);
}

}  // namespace moeq
