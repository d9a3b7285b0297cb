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

// Four lanes hold a block of 32, eight elements each: the block's scale byte
// (the same in all four) and this lane's codes.
__device__ __forceinline__ uint32_t mx4_block(const float (&v)[8], uint32_t* scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t b = mx4_scale_byte(m);
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
            a = __ldg(q);
            if constexpr (kF32) b = __ldg(q + 1);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < (kF32 ? 8 : 4); ++i) {
                if constexpr (kF32) {
                    w[i] = __ldg(static_cast<const uint32_t*>(p) + at + i);
                } else {
                    const uint16_t* h = static_cast<const uint16_t*>(p) + at + 2 * i;
                    w[i] = __ldg(h) | static_cast<uint32_t>(__ldg(h + 1)) << 16;
                }
            }
            a = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (kF32) b = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
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

// A warp's segment of a row: kSegment K blocks of 256 columns, eight of each
// a lane (its loads all issued before the first is used).
constexpr int kSegment = 4;
__host__ __device__ constexpr int segments(int K) { return (mx4_kb(K) + kSegment - 1) / kSegment; }

template <bool kF32, bool kVec, bool kSwiglu>
struct Segment {
    Raw8<kF32> v[kSegment], u[kSwiglu ? kSegment : 1];
    __device__ __forceinline__ void load(const void* x, int64_t row0, int seg, int lane, int K) {
#pragma unroll
        for (int i = 0; i < kSegment; ++i) {
            const int c = (seg * kSegment + i) * kMx4TileCols + lane * 8;
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
        if constexpr (kSwiglu) {
            float g[8];
            u[i].get(g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = swiglu(f[j], g[j]);
        }
        const uint32_t q = mx4_block(f, s);
        if (!in) *s = 0;
        return in ? q : 0u;
    }
};

// The four scale bytes of this lane's 128 columns (lanes 0..15, 16..31).
__device__ __forceinline__ uint32_t scale_word(uint32_t s, int lane) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) word |= __shfl_sync(0xffffffffu, s, (lane & 16) + 4 * j) << (8 * j);
    return word;
}

// Rows of activations, one warp a segment.
template <bool kF32, bool kVec, bool kSwiglu>
__global__ void __launch_bounds__(256) quant_act_kernel(const void* __restrict__ x, int64_t ld, int rows, int K,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    const int lane = threadIdx.x & 31, segs = segments(K);
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t row = item / segs;
    const int seg = static_cast<int>(item - row * segs);
    if (row >= rows) return;
    Segment<kF32, kVec, kSwiglu> g;
    g.load(x, row * ld, seg, lane, K);
#pragma unroll
    for (int i = 0; i < kSegment; ++i) {
        const int kb = seg * kSegment + i, c = kb * kMx4TileCols + lane * 8;
        if (kb * kMx4TileCols >= K) break;
        uint32_t s;
        const uint32_t q = g.quant(i, c < K, &s);
        if (c < K) *reinterpret_cast<uint32_t*>(codes + row * (K >> 1) + (c >> 1)) = q;
        const uint32_t word = scale_word(s, lane);
        if ((lane & 15) == 0)
            *reinterpret_cast<uint32_t*>(scales + row * mx4_scale_pitch(K) + kb * 8 + (lane >> 4) * 4) = word;
    }
}

// Codes and scales back to values.  A value is a code (at most two
// significant bits) times a power of two: exact in bf16 and in fp32 (a
// subnormal of at least 2^-128 fits both).  The scale is applied in two
// halves, because 2^-127 is no normal number.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) dequant_act_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, int rows, int K,
                                                          T* __restrict__ out, int64_t ld) {
    const int lane = threadIdx.x & 31, segs = segments(K);
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
            q[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + row * (K >> 1) + (c >> 1)));
            sc[i] = __ldg(scales + row * mx4_scale_pitch(K) + (c >> 5));
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
// a weight tile, and its row's scale words (lanes 0 and 16 write them).
__device__ __forceinline__ void store_tile(uint8_t* tile, uint8_t* stile, int r, int lane, uint32_t q, uint32_t s) {
    const int chunk = lane >> 2;
    *reinterpret_cast<uint32_t*>(tile + r * 128 + ((chunk ^ (r & 7)) << 4) + (lane & 3) * 4) = q;
    const uint32_t word = scale_word(s, lane);
    if ((lane & 15) == 0)
        *reinterpret_cast<uint32_t*>(stile + (lane >> 4) * 512 + (r & 31) * 16 + (r >> 5) * 4) = word;
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
        const uint32_t q = mx4_block(v, &s);
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
    const int per = plan_rows_per_tile(plan.first[e + 1] - plan.first[e], p.nt);
    const int in_e = r - plan.first[e], t = in_e / per;
    return {static_cast<int64_t>(plan.tile[e] + t) * kb_all, in_e - t * per};
}
// Byte offset, inside a K block's scales, of the word of row `pos` and the
// block's 128-column half `kc`.
__device__ __forceinline__ int scale_at(int pos, int kc, int sb) {
    return kc * (sb >> 1) + (pos >> 7) * 512 + (pos & 31) * 16 + ((pos >> 5) & 3) * 4;
}
__device__ __forceinline__ int act_row(const Mx4Plan& p, int r) {
    return min(p.row_pair ? max(__ldg(p.row_pair + r), 0) / p.top_k : r, p.rows - 1);
}

// From rows to quantise: a warp takes a segment of a row at a time.  The
// first one's loads are issued before the plan is known (they need only the
// row number).
template <bool kF32, bool kVec, bool kSwiglu>
__global__ void __launch_bounds__(kPlanThreads) act_tiles_kernel(RowsIn x, Mx4Plan p, int K, uint8_t* __restrict__ tiles,
                                                                 uint8_t* __restrict__ stiles) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ PlanShared plan;
    const int lane = threadIdx.x & 31, kb_all = mx4_kb(K), segs = segments(K), sb = mx4_tile_scale_bytes(p.nt);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kPlanThreads / 32);
    int64_t it = static_cast<int64_t>(blockIdx.x) * (kPlanThreads / 32) + (threadIdx.x >> 5);
    auto row_of = [&](int64_t i) { return static_cast<int>(i / segs); };
    Segment<kF32, kVec, kSwiglu> g;
    auto load = [&] {
        const int r = row_of(it);
        g.load(x.p, act_row(p, r) * x.ld, static_cast<int>(it - static_cast<int64_t>(r) * segs), lane, K);
    };
    const int64_t most = static_cast<int64_t>(p.R) * segs;
    if (it < most) load();
    plan_scan(p, plan);
    const int64_t items = static_cast<int64_t>(plan.first[p.E]) * segs;
    while (it < items) {
        const int r = row_of(it), seg = static_cast<int>(it - static_cast<int64_t>(r) * segs);
        if (r >= plan.first[0]) {
            const Place at = place_of(plan, p, r, kb_all);
            const int c_at = at.pos * 128 + (((lane >> 2) ^ (at.pos & 7)) << 4) + (lane & 3) * 4;
#pragma unroll
            for (int i = 0; i < kSegment; ++i) {
                const int kb = seg * kSegment + i;
                if (kb >= kb_all) break;
                uint32_t s;
                const uint32_t q = g.quant(i, kb * kMx4TileCols + lane * 8 < K, &s);
                const uint32_t word = scale_word(s, lane);
                *reinterpret_cast<uint32_t*>(tiles + (at.block0 + kb) * p.nt * 128 + c_at) = q;
                if ((lane & 15) == 0)
                    *reinterpret_cast<uint32_t*>(stiles + (at.block0 + kb) * sb + scale_at(at.pos, lane >> 4, sb)) = word;
            }
        }
        it += step;
        if (it < items) load();
    }
}

// From codes: a warp moves a row, 16 bytes of codes and four scale bytes a
// lane at a time.
__global__ void __launch_bounds__(kPlanThreads) code_tiles_kernel(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales, Mx4Plan p, int K,
                                                                  uint8_t* __restrict__ tiles,
                                                                  uint8_t* __restrict__ stiles) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ PlanShared plan;
    plan_scan(p, plan);
    const int lane = threadIdx.x & 31, kb_all = mx4_kb(K), sb = mx4_tile_scale_bytes(p.nt), pitch = mx4_scale_pitch(K);
    const int chunks = K >> 5, all_chunks = kb_all * 8, r_end = plan.first[p.E];
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kPlanThreads / 32);
    for (int64_t r64 = static_cast<int64_t>(blockIdx.x) * (kPlanThreads / 32) + (threadIdx.x >> 5); r64 < r_end;
         r64 += step) {
        const int r = static_cast<int>(r64);
        if (r < plan.first[0]) continue;
        const int64_t row = act_row(p, r);
        const uint4* src = reinterpret_cast<const uint4*>(codes + row * (K >> 1));
        const uint32_t* ssrc = reinterpret_cast<const uint32_t*>(scales + row * pitch);
        const Place at = place_of(plan, p, r, kb_all);
        for (int c0 = 0; c0 < all_chunks; c0 += 128) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * 32 + lane;
                v[i] = c < chunks ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
            }
            const int word = c0 / 4 + lane;  // 32 words of 128 columns for 128 chunks of 32
            const uint32_t w = word * 4 < pitch ? __ldg(ssrc + word) : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * 32 + lane;
                if (c < all_chunks)
                    *reinterpret_cast<uint4*>(tiles + ((at.block0 + (c >> 3)) * p.nt + at.pos) * 128 +
                                              (((c & 7) ^ (at.pos & 7)) << 4)) = v[i];
            }
            if (word * 4 < pitch)
                *reinterpret_cast<uint32_t*>(stiles + (at.block0 + (word >> 1)) * sb + scale_at(at.pos, word & 1, sb)) = w;
        }
    }
}

bool fits(const void* p, int64_t ld, int f32) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (f32 ? 4 : 8) == 0;
}

}  // namespace

cudaError_t launch_mx4_quant_act(RowsIn x, int rows, int K, int act, uint8_t* codes, uint8_t* scales,
                                 cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(rows) * segments(K) + 7) / 8);
    // the second half of a SwiGLU row starts K elements on: K is a multiple of 32
    const bool vec = fits(x.p, x.ld, x.f32);
    auto go = [&](auto kern) {
        kern<<<grid, 256, 0, stream>>>(x.p, x.ld, rows, K, codes, scales);
        return cudaGetLastError();
    };
    if (x.f32) {
        if (act) return vec ? go(quant_act_kernel<true, true, true>) : go(quant_act_kernel<true, false, true>);
        return vec ? go(quant_act_kernel<true, true, false>) : go(quant_act_kernel<true, false, false>);
    }
    if (act) return vec ? go(quant_act_kernel<false, true, true>) : go(quant_act_kernel<false, false, true>);
    return vec ? go(quant_act_kernel<false, true, false>) : go(quant_act_kernel<false, false, false>);
}

cudaError_t launch_mx4_dequant_act(const uint8_t* codes, const uint8_t* scales, int rows, int K, RowsOut out,
                                   cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(rows) * segments(K) + 7) / 8);
    const bool vec = fits(out.p, out.ld, out.f32);
    auto go = [&](auto* o, auto kern) {
        kern<<<grid, 256, 0, stream>>>(codes, scales, rows, K, o, out.ld);
        return cudaGetLastError();
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
    auto grid_of = [&](int64_t warps, int per_sm) {
        const int64_t blocks = (warps + 7) / 8;
        return static_cast<unsigned>(blocks < static_cast<int64_t>(sms) * per_sm ? blocks : sms * per_sm);
    };
    if (src.codes) {
        code_tiles_kernel<<<grid_of(plan.R, 8), kPlanThreads, 0, stream>>>(src.codes, src.scales, plan, K, tiles, stiles);
        return cudaGetLastError();
    }
    const bool vec = fits(src.x.p, src.x.ld, src.x.f32);
    auto go = [&](auto kern) {
        kern<<<grid_of(static_cast<int64_t>(plan.R) * segments(K), 6), kPlanThreads, 0, stream>>>(src.x, plan, K, tiles,
                                                                                               stiles);
        return cudaGetLastError();
    };
    if (src.x.f32) {
        if (src.act) return vec ? go(act_tiles_kernel<true, true, true>) : go(act_tiles_kernel<true, false, true>);
        return vec ? go(act_tiles_kernel<true, true, false>) : go(act_tiles_kernel<true, false, false>);
    }
    if (src.act) return vec ? go(act_tiles_kernel<false, true, true>) : go(act_tiles_kernel<false, false, true>);
    return vec ? go(act_tiles_kernel<false, true, false>) : go(act_tiles_kernel<false, false, false>);
}

}  // namespace moeq
