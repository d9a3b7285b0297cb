// Activations kept in 8 bits between the forward and the backward pass: rows
// to codes and back (also back as the experts' rows), and SwiGLU with its gate
// and up rows kept so, and its gradients from them.
//
// The format is the library's activation quantisation (groups of 1 x 128
// columns, s = fl32(amax / 448), code = RNE(fl32(x / s))) for rows of any
// width: the last group is shorter, and gate and up have groups of their own.
// A value comes back as fl32(code * s), rounded once more to bf16 where that
// is the type.  A group with a NaN or an infinity comes back as NaN.
//
// Each byte moves once: HBM bounds all of them, and the arithmetic of the
// quantisation comes close (see codes8).  Half a warp has a group: eight
// elements a lane, neighbours where rows allow 16-byte accesses (kVec), else
// 16 apart, so that neighbouring lanes still touch neighbouring elements.
#include "moeq_device.cuh"
#include "moeq_rows.h"

namespace moeq {
namespace {

constexpr int kThreads = 256, kHalves = kThreads / 16;  // half warps of a block
constexpr float kNaN = __builtin_nanf("");

// ---------------------------------------------------------- eight elements
// `left`: columns from this lane's first on.
template <bool kVec>
__device__ __forceinline__ int col_of(int lane16) {
    return kVec ? lane16 * 8 : lane16;
}
template <bool kVec>
__device__ __forceinline__ void load8(const float* p, int left, float (&v)[8]) {
    if constexpr (kVec) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (left > 0) {
            a = reinterpret_cast<const float4*>(p)[0];
            b = reinterpret_cast<const float4*>(p)[1];
        }
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 16 * i < left ? p[16 * i] : 0.f;
    }
}
template <bool kVec>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int left, float (&v)[8]) {
    if constexpr (kVec) {
        const uint4 a = left > 0 ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 16 * i < left ? __bfloat162float(p[16 * i]) : 0.f;
    }
}
template <bool kVec>
__device__ __forceinline__ void store8(float* p, int left, const float (&v)[8]) {
    if constexpr (kVec) {
        if (left > 0) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (16 * i < left) p[16 * i] = v[i];
    }
}
template <bool kVec>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int left, const float (&v)[8]) {
    if constexpr (kVec) {
        if (left > 0) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (16 * i < left) p[16 * i] = __float2bfloat16_rn(v[i]);
    }
}
// Eight codes, the first in the lowest byte.
template <bool kVec>
__device__ __forceinline__ uint2 load8(const uint8_t* p, int left) {
    uint2 c = make_uint2(0, 0);
    if constexpr (kVec) {
        if (left > 0) c = *reinterpret_cast<const uint2*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (16 * i < left) c.x |= static_cast<uint32_t>(p[16 * i]) << (8 * i);
            if (16 * (i + 4) < left) c.y |= static_cast<uint32_t>(p[16 * (i + 4)]) << (8 * i);
        }
    }
    return c;
}
template <bool kVec>
__device__ __forceinline__ void store8(uint8_t* p, int left, uint2 c) {
    if constexpr (kVec) {
        if (left > 0) *reinterpret_cast<uint2*>(p) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (16 * i < left) p[16 * i] = static_cast<uint8_t>(c.x >> (8 * i));
            if (16 * (i + 4) < left) p[16 * (i + 4)] = static_cast<uint8_t>(c.y >> (8 * i));
        }
    }
}

// ------------------------------------------------------------ quantisation
__device__ __forceinline__ uint2 pack8(const float (&q)[8]) {
    const auto four = [&](int i) {
        return static_cast<uint32_t>(e4m3x2_from_f32(q[i], q[i + 1])) |
               (static_cast<uint32_t>(e4m3x2_from_f32(q[i + 2], q[i + 3])) << 16);
    };
    return make_uint2(four(0), four(4));
}
// The codes of this lane's eight elements of a group, and its scale.
// Quotients are taken as products with 1 / s, which may be two steps of fp32
// off fl32(x / s): the same code, unless a border between two codes lies that
// near.  Then (8 in 2^20 quotients) the lane divides.  A border is where the
// 20 bits below E4M3's three are 2^19; below 2^-6 the codes are 2^-9 apart, as
// they are in [2^-6, 2^-5), so 2^-6 is added first.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float* scale) {
    uint32_t top = 0;  // as integers, so that a NaN is the largest
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float s = __fdiv_rn(__uint_as_float(top), 448.0f);
    *scale = s;
    if (top >= 0x7F800000u) {
        *scale = kNaN;
        return make_uint2(0, 0);
    }
    float q[8];
    bool near = s < 1e-30f;  // 1 / s may be out of range
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = v[i] * inv;
        const float a = fabsf(q[i]) + (fabsf(q[i]) < 0.015625f ? 0.015625f : 0.f);
        near |= ((__float_as_uint(a) + 0x80004u) & 0xFFFFFu) <= 8u;
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = s == 0.f ? copysignf(0.f, v[i]) : __fdiv_rn(v[i], s);
    }
    return pack8(q);
}
__device__ __forceinline__ void values8(uint2 c, float s, float (&v)[8]) {
    float2 f[4];
    e4m3x4_to_f32(c.x, f[0], f[1]);
    e4m3x4_to_f32(c.y, f[2], f[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = f[i].x * s;
        v[2 * i + 1] = f[i].y * s;
    }
}

// A block's half warps over rows and groups: rows of few groups share a block.
struct Split {
    int log_groups;  // half warps of a row: a power of two, at most kHalves
};
__host__ __device__ constexpr int groups_of(int K) { return (K + kGroup - 1) / kGroup; }
Split split_of(int groups) {
    Split s{0};
    while ((1 << s.log_groups) < groups && (1 << s.log_groups) < kHalves) ++s.log_groups;
    return s;
}
unsigned blocks_of(int rows, Split s) {
    const int per = kHalves >> s.log_groups;
    return static_cast<unsigned>((static_cast<int64_t>(rows) + per - 1) / per);
}
__device__ __forceinline__ int64_t row_of(Split s) {
    const int half = threadIdx.x >> 4;
    return static_cast<int64_t>(blockIdx.x) * (kHalves >> s.log_groups) + (half >> s.log_groups);
}
__device__ __forceinline__ int group_of(Split s) { return (threadIdx.x >> 4) & ((1 << s.log_groups) - 1); }

// ------------------------------------------------------------- rows to codes
// (The shuffles of codes8 want whole warps: rows and groups out of range run
// along with nothing to load or store.)
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const T* x, int64_t ld, int rows, int K, Split sp,
                                                              uint8_t* __restrict__ codes, float* __restrict__ scales) {
    chain();
    const int64_t r = row_of(sp);
    const int G = groups_of(K), g = (blockIdx.y << sp.log_groups) + group_of(sp), lane16 = threadIdx.x & 15;
    const bool live = r < rows && g < G;
    const int c = g * kGroup + col_of<kVec>(lane16), left = live ? min(K, (g + 1) * kGroup) - c : 0;
    float v[8], s;
    load8<kVec>(x + r * ld + c, left, v);
    const uint2 q = codes8(v, &s);
    store8<kVec>(codes + r * K + c, left, q);
    if (live && lane16 == 0) scales[r * G + g] = s;
}

// ------------------------------------------------------------- codes to rows
// xs[pair_row[t, j]] = the values of row t; pair_row NULL: xs[t].  Token-major:
// codes are read once for all their rows.  Rows from offs[E] on are zeroed,
// shared out over the tokens' blocks.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) gather_codes_kernel(const uint8_t* codes, const float* scales, int H, int k,
                                                                const int32_t* offs, int E, int64_t R,
                                                                const int32_t* pair_row, T* __restrict__ xs, int64_t ld) {
    chain();
    const int64_t t = blockIdx.x;
    const int lane16 = threadIdx.x & 15, g = blockIdx.y * (blockDim.x >> 4) + (threadIdx.x >> 4);
    const int c = g * kGroup + col_of<kVec>(lane16), left = min(H, (g + 1) * kGroup) - c;
    if (left <= 0) return;
    float v[8];
    values8(load8<kVec>(codes + t * H + c, left), scales[t * groups_of(H) + g], v);
    if (!pair_row) {
        store8<kVec>(xs + t * ld + c, left, v);
        return;
    }
    for (int j0 = 0; j0 < k; j0 += 8) {
        int r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = j0 + j < k ? pair_row[t * k + j0 + j] : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (r[j] >= 0 && r[j] < R) store8<kVec>(xs + r[j] * ld + c, left, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    for (int64_t r = max(offs[E], 0) + t; r < R; r += gridDim.x) store8<kVec>(xs + r * ld + c, left, v);
}

// ------------------------------------------------------------------- SwiGLU
// 1 / (1 + exp(-g)): at most three steps of fp32 off.
__device__ __forceinline__ float sigmoid(float g) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + expf(-g)));
    return r;
}

struct SwigluArgs {
    int R, I;
    Split sp;
    const int32_t* row_pair;  // [R] or NULL: every row is live
    const float* w;           // [R], a pair's weight, or NULL: 1
};
// Whether a row belongs to an expert, and its pair and weight.
struct RowOf {
    bool live;
    int pair;
    float w;
};
__device__ __forceinline__ RowOf row_info(const SwigluArgs& a, int64_t r) {
    RowOf o{r < a.R, 0, 1.f};
    if (o.live && a.row_pair) {
        o.pair = a.row_pair[r];
        o.live = o.pair >= 0 && o.pair < a.R;
        if (o.live && a.w) o.w = a.w[o.pair];
    }
    return o;
}

// h[r] = w_r silu(gate) up, and gate and up in 8 bits.  A row that belongs to
// no expert is not read; its h, codes and scales are zeros.
template <typename T, bool kVec, bool kKeep>
__global__ void __launch_bounds__(kThreads) swiglu_rows_kernel(const SwigluArgs a, const T* gu, int64_t ld, T* __restrict__ h,
                                                               int64_t ld_h, uint8_t* __restrict__ codes,
                                                               float* __restrict__ scales) {
    chain();
    const int64_t r = row_of(a.sp);
    const int G = groups_of(a.I), g = (blockIdx.y << a.sp.log_groups) + group_of(a.sp), lane16 = threadIdx.x & 15;
    const bool in = r < a.R && g < G;
    const int c = g * kGroup + col_of<kVec>(lane16), left = in ? min(a.I, (g + 1) * kGroup) - c : 0;
    const RowOf row = row_info(a, r);
    const int read = row.live ? left : 0;
    float x[8], u[8], y[8];
    load8<kVec>(gu + r * ld + c, read, x);
    load8<kVec>(gu + r * ld + a.I + c, read, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = row.w * (x[i] * sigmoid(x[i])) * u[i];
    store8<kVec>(h + r * ld_h + c, left, y);
    if constexpr (kKeep) {
        float sx, su;
        const uint2 qx = codes8(x, &sx), qu = codes8(u, &su);
        uint8_t* const at = codes + r * 2 * a.I + c;
        store8<kVec>(at, left, qx);
        store8<kVec>(at + a.I, left, qu);
        if (in && lane16 == 0) {
            scales[r * 2 * G + g] = sx;
            scales[r * 2 * G + G + g] = su;
        }
    }
}

// From the kept rows, p = silu'(gate): d_gate = w dh up p, d_up = w dh silu(gate),
// h again, and d_w[pair] = <dh, silu(gate) up>.  A row's half warps add their
// parts up in a fixed order.  A pair without a row gets d_w 0.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) swiglu_rows_grad_kernel(const SwigluArgs a, const T* dh, int64_t ld_dh,
                                                                    const uint8_t* codes, const float* scales,
                                                                    T* __restrict__ dgu, int64_t ld_dgu, T* __restrict__ h,
                                                                    int64_t ld_h, const int32_t* pair_row,
                                                                    float* __restrict__ dw) {
    chain();
    __shared__ float part[kHalves];
    const int64_t r = row_of(a.sp);
    const int G = groups_of(a.I), lane16 = threadIdx.x & 15;
    const RowOf row = row_info(a, r);
    float dot = 0.f;
    for (int g = group_of(a.sp); g < G && r < a.R; g += 1 << a.sp.log_groups) {
        const int c = g * kGroup + col_of<kVec>(lane16), left = min(a.I, (g + 1) * kGroup) - c;
        const int read = row.live ? left : 0;
        const uint8_t* const at = codes + r * 2 * a.I + c;
        float d[8], x[8], u[8], dx[8], du[8], y[8];
        load8<kVec>(dh + r * ld_dh + c, read, d);
        values8(load8<kVec>(at, read), row.live ? scales[r * 2 * G + g] : 0.f, x);
        values8(load8<kVec>(at + a.I, read), row.live ? scales[r * 2 * G + G + g] : 0.f, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float sig = sigmoid(x[i]), act = x[i] * sig, wd = row.w * d[i];
            dx[i] = wd * u[i] * (sig * (1.f + x[i] * (1.f - sig)));
            du[i] = wd * act;
            y[i] = row.w * act * u[i];
            dot = fmaf(d[i], act * u[i], dot);
        }
        store8<kVec>(dgu + r * ld_dgu + c, left, dx);
        store8<kVec>(dgu + r * ld_dgu + a.I + c, left, du);
        if (h) store8<kVec>(h + r * ld_h + c, left, y);
    }
    if (!dw) return;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane16 == 0) part[threadIdx.x >> 4] = dot;
    __syncthreads();
    if (lane16 == 0 && group_of(a.sp) == 0 && r < a.R) {
        float sum = 0.f;
        for (int i = 0; i < 1 << a.sp.log_groups; ++i) sum += part[(threadIdx.x >> 4) + i];
        if (row.live) dw[row.pair] = sum;
        if (pair_row[r] < 0) dw[r] = 0.f;
    }
}

// Eight neighbours at a time: rows start and step on 16 bytes, codes on 8.
bool fits8(const void* p, int64_t ld, int f32) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (f32 ? 4 : 8) == 0;
}
template <typename F>
cudaError_t by_type(int f32, F f) {
    return f32 ? f(static_cast<float*>(nullptr)) : f(static_cast<__nv_bfloat16*>(nullptr));
}

}  // namespace

cudaError_t launch_fp8_quant_rows(RowsIn x, int rows, int K, uint8_t* codes, float* scales, cudaStream_t stream) {
    const int G = groups_of(K);
    const Split sp = split_of(G);
    const dim3 grid(blocks_of(rows, sp), (G + (1 << sp.log_groups) - 1) >> sp.log_groups);
    const bool vec = K % 8 == 0 && fits8(x.p, x.ld, x.f32);
    return by_type(x.f32, [&](auto* tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        const T* p = static_cast<const T*>(x.p);
        return launch_chained(vec ? quant_rows_kernel<T, true> : quant_rows_kernel<T, false>, grid, kThreads, 0, stream, p,
                              x.ld, rows, K, sp, codes, scales);
    });
}

cudaError_t launch_fp8_gather_rows(const uint8_t* codes, const float* scales, int T, int H, int k, const int32_t* offs,
                                   int E, const int32_t* pair_row, RowsOut xs, cudaStream_t stream) {
    const int G = groups_of(H), threads = G >= kHalves ? kThreads : (G + 1) / 2 * 32;
    const dim3 grid(T, (G * 16 + threads - 1) / threads);
    const bool vec = H % 8 == 0 && fits8(xs.p, xs.ld, xs.f32);
    return by_type(xs.f32, [&](auto* tag) {
        using Ty = std::remove_pointer_t<decltype(tag)>;
        return launch_chained(vec ? gather_codes_kernel<Ty, true> : gather_codes_kernel<Ty, false>, grid, threads, 0, stream,
                              codes, scales, H, k, offs, E, static_cast<int64_t>(T) * k, pair_row, static_cast<Ty*>(xs.p),
                              xs.ld);
    });
}

cudaError_t launch_swiglu_rows(RowsIn gu, int R, int I, const int32_t* row_pair, const float* w, RowsOut h, uint8_t* codes,
                               float* scales, cudaStream_t stream) {
    const int G = groups_of(I);
    const SwigluArgs a = {R, I, split_of(G), row_pair, w};
    const dim3 grid(blocks_of(R, a.sp), (G + (1 << a.sp.log_groups) - 1) >> a.sp.log_groups);
    const bool vec = I % 8 == 0 && fits8(gu.p, gu.ld, gu.f32) && fits8(h.p, h.ld, gu.f32);
    return by_type(gu.f32, [&](auto* tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        auto go = [&](auto kern) {
            return launch_chained(kern, grid, kThreads, 0, stream, a, static_cast<const T*>(gu.p), gu.ld,
                                  static_cast<T*>(h.p), h.ld, codes, scales);
        };
        if (codes) return vec ? go(swiglu_rows_kernel<T, true, true>) : go(swiglu_rows_kernel<T, false, true>);
        return vec ? go(swiglu_rows_kernel<T, true, false>) : go(swiglu_rows_kernel<T, false, false>);
    });
}

cudaError_t launch_swiglu_rows_grad(RowsIn dh, const uint8_t* codes, const float* scales, int R, int I,
                                    const int32_t* row_pair, const float* w, const int32_t* pair_row, RowsOut dgu, RowsOut h,
                                    float* dw, cudaStream_t stream) {
    const SwigluArgs a = {R, I, split_of(groups_of(I)), row_pair, w};
    const bool vec = I % 8 == 0 && fits8(dh.p, dh.ld, dh.f32) && fits8(dgu.p, dgu.ld, dh.f32) &&
                     (!h.p || fits8(h.p, h.ld, dh.f32));
    return by_type(dh.f32, [&](auto* tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        return launch_chained(vec ? swiglu_rows_grad_kernel<T, true> : swiglu_rows_grad_kernel<T, false>,
                              dim3(blocks_of(R, a.sp)), kThreads, 0, stream, a, static_cast<const T*>(dh.p), dh.ld, codes,
                              scales, static_cast<T*>(dgu.p), dgu.ld, static_cast<T*>(h.p), h.ld, pair_row, dw);
    });
}

}  // namespace moeq
