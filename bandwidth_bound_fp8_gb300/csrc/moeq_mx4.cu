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

template <bool kF32, bool kVec>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
    if constexpr (kF32) {
        const float* f = static_cast<const float*>(p) + at;
        if constexpr (kVec) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(f)), b = __ldg(reinterpret_cast<const float4*>(f) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __ldg(f + i);
        }
    } else {
        const __nv_bfloat16* f = static_cast<const __nv_bfloat16*>(p) + at;
        if constexpr (kVec) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(f));
            const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __bfloat162float(__ldg(f + i));
        }
    }
}

// silu(g) * u.  The fast exponential and division are within a few ulp times
// |g|, far below the 4-bit rounding that follows.
__device__ __forceinline__ float swiglu(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

// Rows of activations.  A thread takes eight elements (one or two 16-byte
// loads, four bytes of codes written), four lanes a block.
template <bool kF32, bool kVec, bool kSwiglu>
__global__ void __launch_bounds__(256) quant_act_kernel(const void* __restrict__ x, int64_t ld, int64_t items, int K,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const bool in = item < items;
    const int per_row = K >> 3;
    const int64_t row = in ? item / per_row : 0;
    const int c = in ? static_cast<int>(item - row * per_row) * 8 : 0;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (in) {
        load8<kF32, kVec>(x, row * ld + c, v);
        if constexpr (kSwiglu) {
            float u[8];
            load8<kF32, kVec>(x, row * ld + K + c, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = swiglu(v[i], u[i]);
        }
    }
    uint32_t s;
    const uint32_t q = mx4_block(v, &s);
    if (!in) return;
    *reinterpret_cast<uint32_t*>(codes + row * (K >> 1) + (c >> 1)) = q;
    if ((c & 31) == 0) {
        uint8_t* sr = scales + row * mx4_scale_pitch(K);
        sr[c >> 5] = static_cast<uint8_t>(s);
        if (c + 32 == K)  // the row's scales end on eight bytes
            for (int i = K >> 5; i < mx4_scale_pitch(K); ++i) sr[i] = 0;
    }
}

// Codes and scales back to values.  A value is a code (at most two
// significant bits) times a power of two: exact in bf16 and in fp32 (a
// subnormal of at least 2^-128 fits both).  The scale is applied in two
// halves, because 2^-127 is no normal number.
template <typename T>
__global__ void __launch_bounds__(256) dequant_act_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, int64_t items, int K,
                                                          T* __restrict__ out, int64_t ld, int vec) {
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (item >= items) return;
    const int per_row = K >> 3;
    const int64_t row = item / per_row;
    const int c = static_cast<int>(item - row * per_row) * 8;
    const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(codes + row * (K >> 1) + (c >> 1)));
    const uint32_t s = __ldg(scales + row * mx4_scale_pitch(K) + (c >> 5));
    const int half = (static_cast<int>(s) - 127) >> 1, rest = static_cast<int>(s) - 127 - half;
    const float f0 = pow2_bits(half + 127), f1 = pow2_bits(rest + 127);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t n = (q >> (4 * i)) & 15u;
        const uint32_t m = n & 7u;
        // 0, .5, 1, 1.5, 2, 3, 4, 6: m < 2 has no implicit one
        float a = m < 2 ? 0.5f * m : pow2_bits(126 + static_cast<int>(m >> 1)) * (1.f + 0.5f * (m & 1u));
        a = a * f0 * f1;
        a = s == kNanScale ? __uint_as_float(0x7FFFFFFFu) : a;
        v[i] = (n & 8u) ? -a : a;
    }
    T* o = out + row * ld + c;
    if constexpr (sizeof(T) == 4) {
        if (vec) {
            reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = v[i];
        }
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if (vec) {
            *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float2bfloat16_rn(v[i]);
        }
    }
}

// Where a lane's eight elements of (row r, its 32 lanes = 256 columns) go in
// a weight tile, and its row's scale words (lanes 0 and 16 write them).
__device__ __forceinline__ void store_tile(uint8_t* tile, uint8_t* stile, int r, int lane, uint32_t q, uint32_t s) {
    const int chunk = lane >> 2;
    *reinterpret_cast<uint32_t*>(tile + r * 128 + ((chunk ^ (r & 7)) << 4) + (lane & 3) * 4) = q;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, s, (lane & 16) + 4 * i) << (8 * i);
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
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        const bool in = n < N && c < K;
        if (in) load8<kF32, kVec>(w, (static_cast<int64_t>(e) * N + n) * K + c, v);
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
// so that the product fetches a stage with plain bulk copies.  An item is a
// row's 1024 columns, one warp each; the columns past K of its last block of
// 256 are zeroed (padding rows of a tile are not: they only reach rows of the
// product that are not stored).
constexpr int kSegment = 4;  // K blocks of 256 columns an item

template <int kSrc, bool kVec, bool kSwiglu>  // kSrc: 0 bf16, 1 fp32, 2 codes
__global__ void __launch_bounds__(kPlanThreads) act_tiles_kernel(Mx4Source src, Mx4Plan p, int K,
                                                                 uint8_t* __restrict__ tiles,
                                                                 uint8_t* __restrict__ stiles) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ PlanShared plan;
    plan_scan(p, plan);
    const int lane = threadIdx.x & 31, kb_all = mx4_kb(K), segs = (kb_all + kSegment - 1) / kSegment;
    const int r_end = plan.first[p.E];
    const int64_t items = static_cast<int64_t>(r_end) * segs, step = static_cast<int64_t>(gridDim.x) * (kPlanThreads / 32);
    const int sb = mx4_tile_scale_bytes(p.nt), chunk_bytes = sb / 2;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kPlanThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
        const int r = static_cast<int>(it / segs), seg = static_cast<int>(it - static_cast<int64_t>(r) * segs);
        if (r < plan.first[0]) continue;
        const int a_row = min(p.row_pair ? max(__ldg(p.row_pair + r), 0) / p.top_k : r, p.rows - 1);
        float v[kSegment][8], u[kSegment][8];
        uint32_t q[kSegment], s[kSegment];
#pragma unroll
        for (int i = 0; i < kSegment; ++i) {
            const int c = (seg * kSegment + i) * kMx4TileCols + lane * 8;
            q[i] = s[i] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = u[i][j] = 0.f;
            if (c >= K) continue;
            if constexpr (kSrc == 2) {
                q[i] = __ldg(reinterpret_cast<const uint32_t*>(src.codes + static_cast<int64_t>(a_row) * (K >> 1) + (c >> 1)));
                s[i] = __ldg(src.scales + static_cast<int64_t>(a_row) * mx4_scale_pitch(K) + (c >> 5));
            } else {
                load8<kSrc == 1, kVec>(src.x.p, a_row * src.x.ld + c, v[i]);
                if constexpr (kSwiglu) load8<kSrc == 1, kVec>(src.x.p, a_row * src.x.ld + K + c, u[i]);
            }
        }
        // where the row lies: its expert, tile and place in it
        const int e = plan_find(plan.first, p.E, r);
        const int per = plan_rows_per_tile(plan.first[e + 1] - plan.first[e], p.nt);
        const int in_e = r - plan.first[e], t = in_e / per, pos = in_e - t * per;
        const int64_t block0 = static_cast<int64_t>(plan.tile[e] + t) * kb_all + seg * kSegment;
        const int at = pos * 128 + (((lane >> 2) ^ (pos & 7)) << 4) + (lane & 3) * 4;
        const int s_at = (lane >> 4) * chunk_bytes + (pos >> 7) * 512 + (pos & 31) * 16 + ((pos >> 5) & 3) * 4;
#pragma unroll
        for (int i = 0; i < kSegment; ++i) {
            if (seg * kSegment + i >= kb_all) break;
            if constexpr (kSrc != 2) {
                if constexpr (kSwiglu) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] = swiglu(v[i][j], u[i][j]);
                }
                const bool in = (seg * kSegment + i) * kMx4TileCols + lane * 8 < K;
                q[i] = mx4_block(v[i], &s[i]);
                if (!in) s[i] = 0;
            }
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) word |= __shfl_sync(0xffffffffu, s[i], (lane & 16) + 4 * j) << (8 * j);
            *reinterpret_cast<uint32_t*>(tiles + (block0 + i) * p.nt * 128 + at) = q[i];
            if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(stiles + (block0 + i) * sb + s_at) = word;
        }
    }
}

bool fits(const void* p, int64_t ld, int f32) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (f32 ? 4 : 8) == 0;
}

}  // namespace

cudaError_t launch_mx4_quant_act(RowsIn x, int rows, int K, int act, uint8_t* codes, uint8_t* scales,
                                 cudaStream_t stream) {
    const int64_t items = static_cast<int64_t>(rows) * (K / 8);
    const unsigned grid = static_cast<unsigned>((items + 255) / 256);
    // the second half of a SwiGLU row starts K elements on: K is a multiple of 32
    const bool vec = fits(x.p, x.ld, x.f32);
    auto go = [&](auto kern) {
        kern<<<grid, 256, 0, stream>>>(x.p, x.ld, items, K, codes, scales);
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
    const int64_t items = static_cast<int64_t>(rows) * (K / 8);
    const unsigned grid = static_cast<unsigned>((items + 255) / 256);
    const int vec = fits(out.p, out.ld, out.f32);
    if (out.f32)
        dequant_act_kernel<<<grid, 256, 0, stream>>>(codes, scales, items, K, static_cast<float*>(out.p), out.ld, vec);
    else
        dequant_act_kernel<<<grid, 256, 0, stream>>>(codes, scales, items, K, static_cast<__nv_bfloat16*>(out.p),
                                                     out.ld, vec);
    return cudaGetLastError();
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
    const int segs = (mx4_kb(K) + kSegment - 1) / kSegment;
    const int64_t want = (static_cast<int64_t>(plan.R) * segs + 7) / 8;
    const unsigned grid = static_cast<unsigned>(want < sms * 8 ? want : sms * 8);
    const bool vec = src.codes || fits(src.x.p, src.x.ld, src.x.f32);
    auto go = [&](auto kern) {
        kern<<<grid, kPlanThreads, 0, stream>>>(src, plan, K, tiles, stiles);
        return cudaGetLastError();
    };
    if (src.codes) return go(act_tiles_kernel<2, true, false>);
    if (src.x.f32) {
        if (src.act) return vec ? go(act_tiles_kernel<1, true, true>) : go(act_tiles_kernel<1, false, true>);
        return vec ? go(act_tiles_kernel<1, true, false>) : go(act_tiles_kernel<1, false, false>);
    }
    if (src.act) return vec ? go(act_tiles_kernel<0, true, true>) : go(act_tiles_kernel<0, false, true>);
    return vec ? go(act_tiles_kernel<0, true, false>) : go(act_tiles_kernel<0, false, false>);
}

}  // namespace moeq
