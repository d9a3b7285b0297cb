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
// quantisation comes close.  Half a warp has a group: eight elements a lane,
// neighbours where rows allow 16-byte accesses (kVec), else 16 apart, so that
// neighbouring lanes still touch neighbouring elements.  Measured at 32760 rows
// (floors at the copy rate): SwiGLU of 2 x 2048 bf16 kept in 8 bits 99 us (79),
// its gradient 107 (99); 4095 tokens of 6144 quantised 18 (11), brought back 14
// (11), and as rows 68 (63).
#include "moeq_device.cuh"
#include "moeq_rows.h"

namespace moeq {
namespace {

constexpr int kThreads = 256, kHalves = kThreads / 16;  // half warps of a block
constexpr float kNaN = __builtin_nanf("");

// Two fp32 in a register pair: half the issue slots of their arithmetic, which
// is what these kernels are short of beside HBM.
struct F2 {
    uint64_t b;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.b) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 both(float v) { return f2(v, v); }
__device__ __forceinline__ float lo(F2 a) { return __uint_as_float(static_cast<uint32_t>(a.b)); }
__device__ __forceinline__ float hi(F2 a) { return __uint_as_float(static_cast<uint32_t>(a.b >> 32)); }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(b.b), "l"(c.b));
    return r;
}

// ---------------------------------------------------------- eight elements
// `left`: columns from this lane's first on.
template <bool kVec>
__device__ __forceinline__ int col_of(int lane16) {
    return kVec ? lane16 * 8 : lane16;
}
// As they were read, until they are used.
template <typename T, bool kVec>
struct Eight;
template <bool kVec>
struct Eight<float, kVec> {
    float v[8];
    __device__ __forceinline__ void load(const float* p, int left) {
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
    __device__ __forceinline__ void keep_if(bool live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = live ? v[i] : 0.f;
    }
    __device__ __forceinline__ void get(F2 (&o)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f2(v[2 * i], v[2 * i + 1]);
    }
    // The bits of the largest magnitude (a NaN is the largest).
    __device__ __forceinline__ uint32_t top() const {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        return t;
    }
    // The bytes that start with the signs of elements 4 i .. 4 i + 3.
    __device__ __forceinline__ uint32_t signs(int i) const {
        const uint32_t a = __byte_perm(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), 0x0073);
        return __byte_perm(a, __byte_perm(__float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]), 0x0073), 0x5410);
    }
};
template <bool kVec>
struct Eight<__nv_bfloat16, kVec> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int left) {
        if constexpr (kVec) {
            const uint4 a = left > 0 ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        } else {
            const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 16 * i < left ? q[16 * i] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = v[2 * i] | v[2 * i + 1] << 16;
        }
    }
    __device__ __forceinline__ void keep_if(bool live) {
        const uint32_t mask = live ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] &= mask;
    }
    __device__ __forceinline__ void get(F2 (&o)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    // The same of bf16's 16 bits: two magnitudes a comparison.
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t a = 0x7FFF7FFFu;
        const uint32_t m = __vimax3_u16x2(__vimax3_u16x2(w[0] & a, w[1] & a, w[2] & a), w[3] & a, 0u);
        return max(m & 0xFFFFu, m >> 16);
    }
    __device__ __forceinline__ uint32_t signs(int i) const { return __byte_perm(w[2 * i], w[2 * i + 1], 0x7531); }
};
template <bool kVec>
__device__ __forceinline__ void store8(float* p, int left, const F2 (&v)[4]) {
    if constexpr (kVec) {
        if (left <= 0) return;
        if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {  // a whole sector at once
            asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(v[0].b), "l"(v[1].b), "l"(v[2].b), "l"(v[3].b)
                         : "memory");
        } else {
            reinterpret_cast<float4*>(p)[0] = make_float4(lo(v[0]), hi(v[0]), lo(v[1]), hi(v[1]));
            reinterpret_cast<float4*>(p)[1] = make_float4(lo(v[2]), hi(v[2]), lo(v[3]), hi(v[3]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (16 * i < left) p[16 * i] = i & 1 ? hi(v[i / 2]) : lo(v[i / 2]);
    }
}
template <bool kVec>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int left, const F2 (&v)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo(v[i]), hi(v[i]));
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (kVec) {
        if (left > 0) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        unsigned short* q = reinterpret_cast<unsigned short*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (16 * i < left) q[16 * i] = static_cast<unsigned short>(u[i / 2] >> (16 * (i & 1)));
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
// A group's scale, and 1 / scale in two parts (the first is rounded to
// nearest).  A group that is not finite gets the scale NaN.
struct Scale {
    float s, inv, low;
};
__device__ __forceinline__ Scale scale_of(uint32_t top) {
    const float s = __fdiv_rn(__uint_as_float(top), 448.0f), inv = __frcp_rn(s);
    return {top >= 0x7F800000u ? kNaN : s, inv, fmaf(-s, inv, 1.f) * inv};
}
// Of one group, or of two at once (gate and up), of which each half of the
// half warp's lanes computes one.
template <typename T, bool kVec>
__device__ __forceinline__ Scale scale_one(const Eight<T, kVec>& v) {
    uint32_t top = v.top();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    return scale_of(sizeof(T) == 2 ? top << 16 : top);
}
template <typename T, bool kVec>
__device__ __forceinline__ void scale_two(const Eight<T, kVec>& a, const Eight<T, kVec>& b, Scale& sa, Scale& sb) {
    const int lane = threadIdx.x & 31, first = lane & 16;
    uint32_t ta = a.top(), tb = b.top();
    if constexpr (sizeof(T) == 2) {
        uint32_t t = ta | tb << 16;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) t = __vimax3_u16x2(t, __shfl_xor_sync(0xffffffffu, t, o), 0u);
        ta = t << 16;
        tb = t & 0xFFFF0000u;
    } else {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            ta = max(ta, __shfl_xor_sync(0xffffffffu, ta, o));
            tb = max(tb, __shfl_xor_sync(0xffffffffu, tb, o));
        }
    }
    const Scale m = scale_of(lane & 8 ? tb : ta);
    const auto from = [&](int src) {
        return Scale{__shfl_sync(0xffffffffu, m.s, src), __shfl_sync(0xffffffffu, m.inv, src),
                     __shfl_sync(0xffffffffu, m.low, src)};
    };
    sa = from(first);
    sb = from(first | 8);
}
// The codes of eight elements (v: their values).  A quotient fl32(x / s) is
// x / s from the two parts of 1 / s, at most one step off, corrected by the
// remainder x - q s, which is exact then (P. Markstein, IBM J. Res. Dev. 34,
// 1990, on division by fused multiply-adds).  Ties between codes are common
// where both numbers are bf16 (whenever seven divides amax's significand), so
// an approximate quotient will not do.  A code has its element's sign, zeros
// too.
template <typename T, bool kVec>
__device__ __forceinline__ uint2 codes8(const Eight<T, kVec>& e, const F2 (&v)[4], Scale sc) {
    uint32_t c[4];
    // A remainder's last bit is ulp(q) ulp(s).  Quotients below 2^-11 all have code
    // 0, so from s = 2^-92 on it is 2^-34 2^-115 or more: the smallest fp32.
    if (sc.s < 0x1p-92f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = sc.s == 0.f ? 0u : e4m3x2_from_f32(__fdiv_rn(lo(v[i]), sc.s), __fdiv_rn(hi(v[i]), sc.s));
    } else {
        const F2 inv = both(sc.inv), low = both(sc.low), neg = both(-sc.s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            F2 q = fma2(v[i], inv, v[i] * low);
            q = fma2(fma2(q, neg, v[i]), inv, q);
            c[i] = e4m3x2_from_f32(lo(q), hi(q));
        }
    }
    if (sc.s != sc.s) return make_uint2(0, 0);
    return make_uint2(__byte_perm(c[0], c[1], 0x5410) | (e.signs(0) & 0x80808080u),
                      __byte_perm(c[2], c[3], 0x5410) | (e.signs(1) & 0x80808080u));
}
__device__ __forceinline__ void values8(uint2 c, float s, F2 (&v)[4]) {
    const F2 ss = both(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? c.x : c.y;
        const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(i & 1 ? w >> 16 : w & 0xFFFFu)));
        v[i] = f2(f.x, f.y) * ss;
    }
}

// A block's half warps over rows and groups: rows of few groups share a block.
// Blocks walk down the rows, with the next rows' loads in flight behind this
// one's arithmetic (32760 rows of 2 x 2048 bf16 kept: 99 us so, 126 with a block
// for every row).
struct Split {
    int log_groups;  // half warps of a row: a power of two, at most kHalves
    __device__ __forceinline__ int half() const { return threadIdx.x >> 4; }
    __host__ __device__ int rows() const { return kHalves >> log_groups; }          // of a block at a time
    __device__ __forceinline__ int row() const { return half() >> log_groups; }     // of them, this half warp's
    __device__ __forceinline__ int group() const { return half() & ((1 << log_groups) - 1); }
};
__host__ __device__ constexpr int groups_of(int K) { return (K + kGroup - 1) / kGroup; }
// The most half warps a row, up to 2^most, that leave at most `idle` of them
// without a group in a row's last turn.
Split split_of(int groups, int most, int idle) {
    static_assert(kHalves == 1 << 4, "most is at most 4");
    Split s{most};
    while (((groups + (1 << s.log_groups) - 1) >> s.log_groups << s.log_groups) > groups + idle) --s.log_groups;
    return s;
}
// Where groups are independent, none idle: 32760 bf16 rows of 2 x 1408 (11
// groups, kept) take 73 us with one half warp a row and 115 with 16, of 2 x 2816
// 140 with two and 184, of 2 x 2048 100 with two and 99 with 16.
Split split_of(int groups) { return split_of(groups, 4, 0); }
// Blocks for all rows, at most 16 an SM (four of which run at once) over `wide`
// columns of blocks.  Only accesses of 16 bytes leave registers for loads
// ahead: the others take a block for every few rows.
unsigned blocks_of(int rows, Split s, int wide, bool vec, int sms) {
    const int64_t all = (static_cast<int64_t>(rows) + s.rows() - 1) / s.rows(), most = (16 * sms + wide - 1) / wide;
    return static_cast<unsigned>(all < most || !vec ? all : most);
}

// ------------------------------------------------------------- rows to codes
// (The shuffles of the scale want whole warps: rows and groups out of range run
// along with nothing to load or store.)
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, kVec ? 4 : 5)
    quant_rows_kernel(const T* x, int64_t ld, int rows, int K, Split sp, uint8_t* __restrict__ codes,
                      float* __restrict__ scales) {
    chain();
    const int G = groups_of(K), g = (blockIdx.y << sp.log_groups) + sp.group(), lane16 = threadIdx.x & 15;
    const int c = g * kGroup + col_of<kVec>(lane16), width = min(K, (g + 1) * kGroup) - c;
    const int64_t step = static_cast<int64_t>(gridDim.x) * sp.rows();
    int64_t base = static_cast<int64_t>(blockIdx.x) * sp.rows(), r = base + sp.row();
    Eight<T, kVec> next;
    if (kVec) next.load(x + r * ld + c, r < rows ? width : 0);
    for (; base < rows; base += step, r += step) {
        if (!kVec) next.load(x + r * ld + c, r < rows ? width : 0);
        const Eight<T, kVec> e = next;
        if (kVec) next.load(x + (r + step) * ld + c, r + step < rows ? width : 0);
        F2 v[4];
        e.get(v);
        const Scale s = scale_one(e);
        const bool in = r < rows && g < G;
        store8<kVec>(codes + r * K + c, in ? width : 0, codes8(e, v, s));
        if (in && lane16 == 0) scales[r * G + g] = s.s;
    }
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
    F2 v[4];
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
    for (int i = 0; i < 4; ++i) v[i] = both(0.f);
    for (int64_t r = max(offs[E], 0) + t; r < R; r += gridDim.x) store8<kVec>(xs + r * ld + c, left, v);
}

// ------------------------------------------------------------------- SwiGLU
// 1 / (1 + exp(-g)), also where that is below 2^-126: silu and its products with
// large numbers are not.  exp(-g) and 1 / (1 + exp(-g)) would leave fp32's normal
// numbers there; t / (1 + t), t = exp(g), does not (and t is subnormal where the
// sigmoid is).  For fp32 rows at most four steps off.  For bf16 rows exp(-g) is
// 2^(-g log2 e) of the rounded product: |g| steps more, which half a step of bf16
// (2^15 of fp32's) does not show.  (A choice for eight gates at once: 32760 rows
// of 2048, the gradient in bf16 107 us, by t / (1 + t) alone 111.)
template <typename T>
__device__ __forceinline__ void sigmoids(const F2 (&g)[4], F2 (&o)[4]) {
    float least = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) least = fminf(least, fminf(lo(g[i]), hi(g[i])));
    if (least >= -80.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t[2], r[2];
            if constexpr (sizeof(T) == 2) {
                const F2 e = g[i] * both(-1.44269504f);
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t[0]) : "f"(lo(e)));
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t[1]) : "f"(hi(e)));
            } else {
                t[0] = expf(-lo(g[i]));
                t[1] = expf(-hi(g[i]));
            }
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[0]) : "f"(1.f + t[0]));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[1]) : "f"(1.f + t[1]));
            o[i] = f2(r[0], r[1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float r[2];
            const float t = expf(-fabsf(lo(g[i]))), u = expf(-fabsf(hi(g[i])));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[0]) : "f"(1.f + t));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[1]) : "f"(1.f + u));
            o[i] = f2(lo(g[i]) < 0.f ? t : 1.f, hi(g[i]) < 0.f ? u : 1.f) * f2(r[0], r[1]);
        }
    }
}
// For outputs in the rows' type alone.  bf16: 2^-24 / (2^-24 + 2^(-g log2 e - 24))
// is normal throughout, and its exponent's rounding (17 steps) does not show
// either.  (The forward pass is short of issue slots: the same rows kept in 8 bits
// 99 us so and 100.5 with a choice; 97.5 with the sigmoid cut off at 2^-126.)
template <typename T>
__device__ __forceinline__ void sigmoids_out(const F2 (&g)[4], F2 (&o)[4]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t[2], r[2];
            const F2 e = fma2(g[i], both(-1.44269504f), both(-24.f));
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t[0]) : "f"(lo(e)));
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t[1]) : "f"(hi(e)));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[0]) : "f"(0x1p-24f + t[0]));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[1]) : "f"(0x1p-24f + t[1]));
            o[i] = f2(r[0], r[1]) * both(0x1p-24f);
        }
    } else {
        sigmoids<T>(g, o);
    }
}

struct SwigluArgs {
    int R, I;
    Split sp;
    const int32_t* row_pair;  // [R] or NULL: every row is live
    const float* w;           // [R], a pair's weight, or NULL: 1
};
// A row's pair; -1 where it belongs to no expert (or is none).
__device__ __forceinline__ int pair_of(const SwigluArgs& a, int64_t r) {
    if (r >= a.R) return -1;
    if (!a.row_pair) return 0;
    const int pair = a.row_pair[r];
    return pair < a.R ? pair : -1;
}
__device__ __forceinline__ float weight_of(const SwigluArgs& a, int pair) { return a.w && pair >= 0 ? a.w[pair] : 1.f; }

// h[r] = w_r silu(gate) up, and gate and up in 8 bits.  The h, codes and scales
// of a row that belongs to no expert are zeros, whatever it holds.
template <typename T, bool kVec, bool kKeep>
__global__ void __launch_bounds__(kThreads, kVec ? 4 : 5)
    swiglu_rows_kernel(const SwigluArgs a, const T* gu, int64_t ld, T* __restrict__ h, int64_t ld_h,
                       uint8_t* __restrict__ codes, float* __restrict__ scales) {
    chain();
    const int G = groups_of(a.I), g = (blockIdx.y << a.sp.log_groups) + a.sp.group(), lane16 = threadIdx.x & 15;
    const int c = g * kGroup + col_of<kVec>(lane16), width = min(a.I, (g + 1) * kGroup) - c;
    const int64_t step = static_cast<int64_t>(gridDim.x) * a.sp.rows();
    int64_t base = static_cast<int64_t>(blockIdx.x) * a.sp.rows(), r = base + a.sp.row();
    Eight<T, kVec> next_x, next_u;
    int next_pair;
    auto fetch = [&](int64_t row) {
        const int left = row < a.R ? width : 0;
        next_x.load(gu + row * ld + c, left);
        next_u.load(gu + row * ld + a.I + c, left);
        next_pair = pair_of(a, row);
    };
    if (kVec) fetch(r);
    for (; base < a.R; base += step, r += step) {
        if (!kVec) fetch(r);
        Eight<T, kVec> ex = next_x, eu = next_u;
        const int pair = next_pair;
        const float w = weight_of(a, pair);
        if (kVec) fetch(r + step);
        ex.keep_if(pair >= 0);
        eu.keep_if(pair >= 0);
        F2 x[4], u[4], y[4];
        ex.get(x);
        eu.get(u);
        const bool in = r < a.R && g < G;
        const int left = in ? width : 0;
        if constexpr (kKeep) {
            Scale sx, su;
            scale_two(ex, eu, sx, su);
            uint8_t* const at = codes + r * 2 * a.I + c;
            store8<kVec>(at, left, codes8(ex, x, sx));
            store8<kVec>(at + a.I, left, codes8(eu, u, su));
            if (in && lane16 == 0) {
                scales[r * 2 * G + g] = sx.s;
                scales[r * 2 * G + G + g] = su.s;
            }
        }
        F2 sig[4];
        sigmoids_out<T>(x, sig);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = both(w) * (x[i] * sig[i]) * u[i];
        store8<kVec>(h + r * ld_h + c, left, y);
    }
}

// From the kept rows, p = silu'(gate): d_gate = w dh up p, d_up = w dh silu(gate),
// h again, and d_w[pair] = <dh, silu(gate) up>.  A row's half warps add their
// parts up in a fixed order.  A pair without a row gets d_w 0.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 4)
    swiglu_rows_grad_kernel(const SwigluArgs a, const T* dh, int64_t ld_dh, const uint8_t* codes, const float* scales,
                            T* __restrict__ dgu, int64_t ld_dgu, T* __restrict__ h, int64_t ld_h,
                            const int32_t* pair_row, float* __restrict__ dw) {
    chain();
    __shared__ float part[2][kHalves];
    const int G = groups_of(a.I), g0 = a.sp.group(), lane16 = threadIdx.x & 15;
    const int64_t step = static_cast<int64_t>(gridDim.x) * a.sp.rows();
    int64_t base = static_cast<int64_t>(blockIdx.x) * a.sp.rows(), r = base + a.sp.row();
    Eight<T, kVec> next_d;
    uint2 next_x, next_u;
    float next_sx, next_su;
    int next_pair;
    auto width_of = [&](int g) { return min(a.I, (g + 1) * kGroup) - g * kGroup - col_of<kVec>(lane16); };
    auto fetch = [&](int64_t row, int g) {
        const int c = g * kGroup + col_of<kVec>(lane16);
        const bool in = row < a.R && g < G;
        const int left = in ? width_of(g) : 0;
        const uint8_t* const at = codes + row * 2 * a.I + c;
        next_d.load(dh + row * ld_dh + c, left);
        next_x = load8<kVec>(at, left);
        next_u = load8<kVec>(at + a.I, left);
        next_sx = in ? scales[row * 2 * G + g] : 0.f;
        next_su = in ? scales[row * 2 * G + G + g] : 0.f;
        next_pair = pair_of(a, row);
    };
    if (kVec) fetch(r, g0);
    for (int turn = 0; base < a.R; base += step, r += step, turn ^= 1) {
        const int pair = kVec ? next_pair : pair_of(a, r);
        const float w = weight_of(a, pair);
        F2 dot = both(0.f);
        for (int gb = 0; gb < G; gb += 1 << a.sp.log_groups) {
            const int g = gb + g0, c = g * kGroup + col_of<kVec>(lane16);
            const int left = r < a.R && g < G ? width_of(g) : 0;
            if (!kVec) fetch(r, g);
            Eight<T, kVec> ed = next_d;
            uint2 cx = next_x, cu = next_u;
            float sx = next_sx, su = next_su;
            const bool last = gb + (1 << a.sp.log_groups) >= G;
            if (kVec) fetch(last ? r + step : r, last ? g0 : g + (1 << a.sp.log_groups));
            if (pair < 0) {
                cx = cu = make_uint2(0, 0);
                sx = su = 0.f;
            }
            ed.keep_if(pair >= 0);
            F2 d[4], x[4], u[4], dx[4], du[4], y[4];
            ed.get(d);
            values8(cx, sx, x);
            values8(cu, su, u);
            const F2 one = both(1.f), minus = both(-1.f), ww = both(w);
            F2 s[4];
            sigmoids<T>(x, s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 sig = s[i], act = x[i] * sig, da = d[i] * act, wu = ww * u[i];
                dot = fma2(da, u[i], dot);
                du[i] = da * ww;
                y[i] = act * wu;
                dx[i] = d[i] * wu * (sig * fma2(x[i], fma2(sig, minus, one), one));
            }
            store8<kVec>(dgu + r * ld_dgu + c, left, dx);
            store8<kVec>(dgu + r * ld_dgu + a.I + c, left, du);
            if (h) store8<kVec>(h + r * ld_h + c, left, y);
        }
        if (!dw) continue;
        float all = lo(dot) + hi(dot);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        if (a.sp.log_groups == 1) {
            all += __shfl_xor_sync(0xffffffffu, all, 16);
        } else if (a.sp.log_groups > 1) {
            if (lane16 == 0) part[turn][a.sp.half()] = all;
            __syncthreads();  // (one a row: the other turn's parts are read before the next)
            if (g0 == 0) {
                all = 0.f;
                for (int i = 0; i < 1 << a.sp.log_groups; ++i) all += part[turn][a.sp.half() + i];
            }
        }
        if (lane16 == 0 && g0 == 0 && r < a.R) {
            if (pair >= 0) dw[pair] = all;
            if (pair_row[r] < 0) dw[r] = 0.f;
        }
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

cudaError_t launch_fp8_quant_rows(RowsIn x, int rows, int K, uint8_t* codes, float* scales, int sms, cudaStream_t stream) {
    const int G = groups_of(K);
    const Split sp = split_of(G);
    const int wide = (G + (1 << sp.log_groups) - 1) >> sp.log_groups;
    const bool vec = K % 8 == 0 && fits8(x.p, x.ld, x.f32);
    const dim3 grid(blocks_of(rows, sp, wide, vec, sms), wide);
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
                               float* scales, int sms, cudaStream_t stream) {
    const int G = groups_of(I);
    const SwigluArgs a = {R, I, split_of(G), row_pair, w};
    const int wide = (G + (1 << a.sp.log_groups) - 1) >> a.sp.log_groups;
    const bool vec = I % 8 == 0 && fits8(gu.p, gu.ld, gu.f32) && fits8(h.p, h.ld, gu.f32);
    const dim3 grid(blocks_of(R, a.sp, wide, vec, sms), wide);
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
                                    float* dw, int sms, cudaStream_t stream) {
    const bool vec = I % 8 == 0 && fits8(dh.p, dh.ld, dh.f32) && fits8(dgu.p, dgu.ld, dh.f32) &&
                     (!h.p || fits8(h.p, h.ld, dh.f32));
    // A warp a row where there are rows enough: its part of d_w then needs no
    // barrier (32760 bf16 rows of 2048: 108 us, 117 with half a block a row and 128
    // with a block; of 1001: 83, 101 and 100).  Half a block otherwise (2048 rows of
    // 4096: 15.4, 16.4 with a block, 22.9 with a warp), a block where rows are fewer
    // than SMs.
    const int G = groups_of(I), most = R >= 96 * sms ? 1 : R > sms ? 3 : 4;
    const SwigluArgs a = {R, I, split_of(G, most, G / 10), row_pair, w};
    return by_type(dh.f32, [&](auto* tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        return launch_chained(vec ? swiglu_rows_grad_kernel<T, true> : swiglu_rows_grad_kernel<T, false>,
                              dim3(blocks_of(R, a.sp, 1, vec, sms)), kThreads, 0, stream, a, static_cast<const T*>(dh.p),
                              dh.ld, codes, scales, static_cast<T*>(dgu.p), dgu.ld, static_cast<T*>(h.p), h.ld, pair_row, dw);
    });
}

}  // namespace moeq
