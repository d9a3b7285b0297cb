// C ABI entry points of the operators that take any number of tokens
// (include/moeq.h): argument checks on the host, then the launches.
#include <atomic>

#include "moeq_rows.h"

using namespace moeq;

namespace {

struct Device {
    bool ok = false;
    int sms = 0;
};

// (No lock and no container: nothing here may throw through a C entry.)
Device current_device() {
    static std::atomic<int> known[128];  // the SM count of a device that runs this, -1 of another; 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return Device{};
    }
    const bool keep = dev >= 0 && dev < 128;
    int sms = keep ? known[dev].load(std::memory_order_relaxed) : 0;
    if (!sms) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return Device{};
        }
        if (major != 10 || minor != 3) sms = -1;
        if (keep) known[dev].store(sms, std::memory_order_relaxed);
    }
    return sms > 0 ? Device{true, sms} : Device{};
}

constexpr int64_t kMaxPairs = int64_t(1) << 30;  // T * top_k and R: row numbers stay in 31 bits
constexpr int kMaxWidth = 1 << 20;               // H and N
// Rows of a gathered product from which the activations are quantised once,
// in token order, and their codes gathered; below, each row is quantised as
// it is gathered (one launch less, top_k times the arithmetic).  With a product
// narrow enough to show it (N = 128, 8 experts), K = 6144 and top-8: 2048 rows
// take 21.5 us once and 21.0 as they are gathered, 4096 rows 24.0 and 27.2,
// 65536 rows 137 and 243; K = 2048 and top-2: 4096 rows 16.9 and 16.0, 8192
// rows 20.5 and 22.4.
constexpr int kQuantOnceRows = 4096;

inline bool al(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool type_ok(moeq_dtype t) { return t == MOEQ_BF16 || t == MOEQ_F32; }
inline size_t size_of(moeq_dtype t) { return t == MOEQ_F32 ? 4 : 2; }
inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
inline moeq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOEQ_OK : MOEQ_ERR_CUDA; }
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Tokens, slots and experts of the routing calls.
bool slots_ok(int T, int top_k, int E) {
    return T >= 0 && top_k >= 1 && top_k <= MOEQ_MAX_TOPK && E >= 1 && E <= MOEQ_MAX_EXPERTS &&
           static_cast<int64_t>(T) * top_k <= kMaxPairs;
}
// A matrix of rows at least `width` apart, on its elements' alignment.
bool rows_ok(const void* p, moeq_dtype t, int64_t ld, int64_t width) {
    return type_ok(t) && al(p, size_of(t)) && ld >= width;
}

// A product's workspace: the header (status word), the tickets of units cut
// between CTAs, row-major codes and scales (rows quantised once before they
// are gathered), the token tiles and their scales, and the parts' sums.
struct Mx4Ws {
    size_t tickets, codes, scales, tiles, stiles, part, end;
    Mx4Tiling tiling;
};
Mx4Ws mx4_ws(int64_t rows, int K, int E, int R, int sms) {
    Mx4Ws l;
    l.tiling = mx4_tiling(R > 0 ? R : 1, E);
    const int nt = l.tiling.nt;
    const size_t blocks = static_cast<size_t>(mx4_max_tiles(R > 0 ? R : 1, E, nt)) * mx4_kb(K);
    l.tickets = 256;
    l.codes = l.tickets + up256(kMx4Tickets * sizeof(int));
    l.scales = l.codes + up256(static_cast<size_t>(rows) * (K / 2));
    l.tiles = l.scales + up256(static_cast<size_t>(rows) * mx4_scale_pitch(K));
    l.stiles = l.tiles + up256(blocks * nt * 128);
    l.part = l.stiles + up256(blocks * mx4_tile_scale_bytes(nt));
    l.end = l.part + static_cast<size_t>(sms) * nt * 128 * sizeof(float);
    return l;
}

bool mx4_shape_ok(int K, int N) { return K >= 32 && K % 32 == 0 && K <= MOEQ_MAX_K && N >= 1 && N <= kMaxWidth; }

}  // namespace

extern "C" {

moeq_status moeq_route_rows(const float* logits, int64_t ld, int T, int E, int top_k, int32_t* topk_id, float* topk_w,
                            void* stream) {
    if (!slots_ok(T, top_k, E) || top_k > E) return MOEQ_ERR_INVALID_ARG;
    if (T == 0) return MOEQ_OK;
    if (!rows_ok(logits, MOEQ_F32, ld, E) || !al(topk_id, 4) || !al(topk_w, 4)) return MOEQ_ERR_INVALID_ARG;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    return cuda_status(launch_route_rows(logits, ld, T, E, top_k, topk_id, topk_w, as_stream(stream)));
}

moeq_status moeq_route_rows_grad(const float* d_topk_w, const int32_t* topk_id, const float* topk_w, int T, int E,
                                 int top_k, float* d_logits, int64_t ld, void* stream) {
    if (!slots_ok(T, top_k, E) || top_k > E) return MOEQ_ERR_INVALID_ARG;
    if (T == 0) return MOEQ_OK;
    if (!rows_ok(d_logits, MOEQ_F32, ld, E) || !al(d_topk_w, 4) || !al(topk_id, 4) || !al(topk_w, 4))
        return MOEQ_ERR_INVALID_ARG;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    return cuda_status(launch_route_rows_grad(d_topk_w, topk_id, topk_w, T, E, top_k, d_logits, ld, as_stream(stream)));
}

moeq_status moeq_expert_sort(const int32_t* topk_id, int T, int top_k, int E, int32_t* offs, int32_t* pair_row,
                             int32_t* row_pair, void* stream) {
    if (!slots_ok(T, top_k, E) || !al(offs, 4)) return MOEQ_ERR_INVALID_ARG;
    if (T > 0 && (!al(topk_id, 4) || !al(pair_row, 4) || !al(row_pair, 4))) return MOEQ_ERR_INVALID_ARG;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    return cuda_status(launch_expert_sort(topk_id, T, top_k, E, offs, pair_row, row_pair, as_stream(stream)));
}

moeq_status moeq_gather_rows(const void* x, moeq_dtype dtype, int64_t ld_x, int T, int H, int top_k,
                             const int32_t* offs, int E, const int32_t* pair_row, void* xs, int64_t ld_xs,
                             void* stream) {
    if (!slots_ok(T, top_k, E) || !type_ok(dtype)) return MOEQ_ERR_INVALID_ARG;
    if (H < 1 || H > kMaxWidth) return MOEQ_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOEQ_OK;
    if (!rows_ok(x, dtype, ld_x, H) || !rows_ok(xs, dtype, ld_xs, H) || !al(offs, 4) || !al(pair_row, 4))
        return MOEQ_ERR_INVALID_ARG;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    const int f32 = dtype == MOEQ_F32;
    return cuda_status(launch_gather_rows({x, ld_x, f32}, T, H, top_k, offs, E, pair_row, {xs, ld_xs, f32},
                                          as_stream(stream)));
}

moeq_status moeq_combine_rows(const void* y, moeq_dtype y_dtype, int64_t ld_y, int T, int H, int top_k,
                              const int32_t* pair_row, const float* topk_w, const void* base_opt, int64_t ld_base,
                              void* out, moeq_dtype out_dtype, int64_t ld_out, void* stream) {
    if (!slots_ok(T, top_k, 1) || !type_ok(y_dtype) || !type_ok(out_dtype)) return MOEQ_ERR_INVALID_ARG;
    if (H < 1 || H > kMaxWidth) return MOEQ_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOEQ_OK;
    if (!rows_ok(y, y_dtype, ld_y, H) || !rows_ok(out, out_dtype, ld_out, H) || !al(pair_row, 4) || !al(topk_w, 4) ||
        (base_opt && !rows_ok(base_opt, out_dtype, ld_base, H)))
        return MOEQ_ERR_INVALID_ARG;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    const int of = out_dtype == MOEQ_F32;
    return cuda_status(launch_combine_rows({y, ld_y, y_dtype == MOEQ_F32}, T, H, top_k, pair_row, topk_w,
                                           {base_opt, ld_base, of}, {out, ld_out, of}, as_stream(stream)));
}

moeq_status moeq_gather_rows_grad(const void* d_xs, moeq_dtype dtype, int64_t ld_xs, int T, int H, int top_k,
                                  const int32_t* pair_row, void* d_x, int64_t ld_x, void* stream) {
    if (!slots_ok(T, top_k, 1) || !type_ok(dtype)) return MOEQ_ERR_INVALID_ARG;
    if (H < 1 || H > kMaxWidth) return MOEQ_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOEQ_OK;
    if (!rows_ok(d_xs, dtype, ld_xs, H) || !rows_ok(d_x, dtype, ld_x, H) || !al(pair_row, 4))
        return MOEQ_ERR_INVALID_ARG;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    const int f32 = dtype == MOEQ_F32;
    return cuda_status(launch_combine_rows({d_xs, ld_xs, f32}, T, H, top_k, pair_row, nullptr, {nullptr, 0, f32},
                                           {d_x, ld_x, f32}, as_stream(stream)));
}

moeq_status moeq_combine_rows_grad(const void* d_out, moeq_dtype out_dtype, int64_t ld_out, const void* y,
                                   moeq_dtype y_dtype, int64_t ld_y, int T, int H, int top_k, const int32_t* offs,
                                   int E, const int32_t* pair_row, const float* topk_w, void* d_y, int64_t ld_dy,
                                   float* d_topk_w, void* stream) {
    if (!slots_ok(T, top_k, E) || !type_ok(y_dtype) || !type_ok(out_dtype)) return MOEQ_ERR_INVALID_ARG;
    if (H < 1 || H > kMaxWidth) return MOEQ_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOEQ_OK;
    if (!rows_ok(d_out, out_dtype, ld_out, H) || !rows_ok(y, y_dtype, ld_y, H) || !rows_ok(d_y, y_dtype, ld_dy, H) ||
        !al(offs, 4) || !al(pair_row, 4) || !al(topk_w, 4) || !al(d_topk_w, 4))
        return MOEQ_ERR_INVALID_ARG;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    const int yf = y_dtype == MOEQ_F32;
    return cuda_status(launch_combine_rows_grad({d_out, ld_out, out_dtype == MOEQ_F32}, {y, ld_y, yf}, T, H, top_k,
                                                offs, E, pair_row, topk_w, {d_y, ld_dy, yf}, d_topk_w,
                                                as_stream(stream)));
}

int moeq_mx4_scale_pitch(int K) { return K >= 32 && K % 32 == 0 && K <= MOEQ_MAX_K ? mx4_scale_pitch(K) : 0; }

size_t moeq_mx4_weight_bytes(int E, int N, int K) {
    if (E < 1 || E > 65535 || !mx4_shape_ok(K, N)) return 0;
    return static_cast<size_t>(E) * mx4_nb(N) * mx4_kb(K) * kMx4TileBytes;
}

size_t moeq_mx4_weight_scale_bytes(int E, int N, int K) { return moeq_mx4_weight_bytes(E, N, K) / 16; }

moeq_status moeq_mx4_quant_act(const void* x, moeq_dtype dtype, int64_t ld, int rows, int K, moeq_act act,
                               uint8_t* codes, uint8_t* scales, void* stream) {
    if (rows < 0 || !type_ok(dtype) || (act != MOEQ_ACT_NONE && act != MOEQ_ACT_SWIGLU)) return MOEQ_ERR_INVALID_ARG;
    if (!mx4_shape_ok(K, 1)) return MOEQ_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return MOEQ_OK;
    if (!rows_ok(x, dtype, ld, act == MOEQ_ACT_SWIGLU ? 2 * static_cast<int64_t>(K) : K) || !al(codes, 16) ||
        !al(scales, 16))
        return MOEQ_ERR_INVALID_ARG;
    const Device dev = current_device();
    if (!dev.ok) return MOEQ_ERR_DEVICE;
    return cuda_status(launch_mx4_quant_act({x, ld, dtype == MOEQ_F32}, rows, K, act, codes, scales, dev.sms,
                                            as_stream(stream)));
}

moeq_status moeq_mx4_dequant_act(const uint8_t* codes, const uint8_t* scales, int rows, int K, void* out,
                                 moeq_dtype dtype, int64_t ld, void* stream) {
    if (rows < 0 || !type_ok(dtype)) return MOEQ_ERR_INVALID_ARG;
    if (!mx4_shape_ok(K, 1)) return MOEQ_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return MOEQ_OK;
    if (!rows_ok(out, dtype, ld, K) || !al(codes, 16) || !al(scales, 16)) return MOEQ_ERR_INVALID_ARG;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    return cuda_status(launch_mx4_dequant_act(codes, scales, rows, K, {out, ld, dtype == MOEQ_F32}, as_stream(stream)));
}

moeq_status moeq_mx4_quant_weight(const void* w, moeq_dtype dtype, int E, int N, int K, uint8_t* tiles,
                                  uint8_t* scale_tiles, void* stream) {
    if (E < 1 || E > 65535 || !type_ok(dtype) || !al(w, size_of(dtype)) || !al(tiles, 16) || !al(scale_tiles, 16))
        return MOEQ_ERR_INVALID_ARG;
    if (!mx4_shape_ok(K, N)) return MOEQ_ERR_UNSUPPORTED_SHAPE;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    return cuda_status(launch_mx4_quant_weight(w, dtype == MOEQ_F32, E, N, K, tiles, scale_tiles, as_stream(stream)));
}

moeq_status moeq_mx4_pack_weight(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, uint8_t* tiles,
                                 uint8_t* scale_tiles, void* stream) {
    if (E < 1 || E > 65535 || !al(codes, 16) || !al(scales, 1) || !al(tiles, 16) || !al(scale_tiles, 16))
        return MOEQ_ERR_INVALID_ARG;
    if (!mx4_shape_ok(K, N)) return MOEQ_ERR_UNSUPPORTED_SHAPE;
    if (!current_device().ok) return MOEQ_ERR_DEVICE;
    return cuda_status(launch_mx4_pack_weight(codes, scales, E, N, K, tiles, scale_tiles, as_stream(stream)));
}

size_t moeq_mx4_expert_gemm_workspace_size(int rows, int K, int N, int E, int R) {
    const Device dev = current_device();
    if (!dev.ok || rows < 0 || R < 0 || R > kMaxPairs || E < 1 || E > MOEQ_MAX_EXPERTS || !mx4_shape_ok(K, N)) return 0;
    return mx4_ws(rows, K, E, R, dev.sms).end;
}

moeq_status moeq_mx4_expert_gemm(const void* x, moeq_dtype x_dtype, int64_t ld_x, const uint8_t* x_scales, int rows,
                                 int K, moeq_act act, const uint8_t* w, const uint8_t* w_scales, int N,
                                 const int32_t* offs, int E, int R, const int32_t* row_pair_opt, int top_k, void* y,
                                 moeq_dtype y_dtype, int64_t ld_y, void* ws, size_t ws_bytes, void* stream) {
    const bool codes_in = x_dtype == MOEQ_MX4;
    if (rows < 0 || R < 0 || R > kMaxPairs || E < 1 || E > MOEQ_MAX_EXPERTS || top_k < 1 || top_k > MOEQ_MAX_TOPK ||
        !type_ok(y_dtype) || (!codes_in && !type_ok(x_dtype)) || (act != MOEQ_ACT_NONE && act != MOEQ_ACT_SWIGLU) ||
        (codes_in && act != MOEQ_ACT_NONE) || codes_in != (x_scales != nullptr))
        return MOEQ_ERR_INVALID_ARG;
    if (!mx4_shape_ok(K, N)) return MOEQ_ERR_UNSUPPORTED_SHAPE;
    // the copies count rows of 128 bytes in 31 bits: 256 GiB of tiles
    const int nt = mx4_tiling(R > 0 ? R : 1, E).nt;
    if (static_cast<int64_t>(E) * mx4_nb(N) * mx4_kb(K) >= (int64_t(1) << 24) ||
        mx4_max_tiles(R > 0 ? R : 1, E, nt) * nt * mx4_kb(K) >= (int64_t(1) << 31))
        return MOEQ_ERR_UNSUPPORTED_SHAPE;
    // without an index row r reads activation row r; with rows to fill there has to be one to read
    if ((!row_pair_opt && rows < R) || (R > 0 && rows == 0)) return MOEQ_ERR_INVALID_ARG;
    if (R == 0) return MOEQ_OK;
    if (codes_in ? (!al(x, 16) || !al(x_scales, 16))
                 : !rows_ok(x, x_dtype, ld_x, act == MOEQ_ACT_SWIGLU ? 2 * static_cast<int64_t>(K) : K))
        return MOEQ_ERR_INVALID_ARG;
    if (!al(w, 16) || !al(w_scales, 16) || !al(offs, 4) || (row_pair_opt && !al(row_pair_opt, 4)) ||
        !rows_ok(y, y_dtype, ld_y, N))
        return MOEQ_ERR_INVALID_ARG;
    const Device dev = current_device();
    if (!dev.ok) return MOEQ_ERR_DEVICE;
    const Mx4Ws l = mx4_ws(codes_in ? 0 : rows, K, E, R, dev.sms);
    if (!al(ws, 16) || ws_bytes < l.end) return MOEQ_ERR_WORKSPACE;
    uint8_t* u8 = static_cast<uint8_t*>(ws);
    cudaStream_t st = as_stream(stream);
    Mx4Source src = {{x, ld_x, x_dtype == MOEQ_F32}, act, nullptr, nullptr};
    if (codes_in) {
        src.codes = static_cast<const uint8_t*>(x);
        src.scales = x_scales;
    } else if (row_pair_opt && R >= kQuantOnceRows && rows < R) {
        src.codes = u8 + l.codes;
        src.scales = u8 + l.scales;
        if (launch_mx4_quant_act(src.x, rows, K, act, u8 + l.codes, u8 + l.scales, dev.sms, st) != cudaSuccess)
            return MOEQ_ERR_CUDA;
    }
    Mx4GemmArgs a = {};
    a.plan = {offs, row_pair_opt, E, R, top_k, rows, l.tiling.nt, l.tiling.align};
    if (launch_mx4_act_tiles(src, a.plan, K, u8 + l.tiles, u8 + l.stiles, dev.sms, st) != cudaSuccess)
        return MOEQ_ERR_CUDA;
    a.w = w;
    a.sw = w_scales;
    a.a = u8 + l.tiles;
    a.sa = u8 + l.stiles;
    a.y = y;
    a.ld_y = ld_y;
    a.y_f32 = y_dtype == MOEQ_F32;
    a.K = K;
    a.N = N;
    a.status = reinterpret_cast<int*>(u8);
    a.tickets = reinterpret_cast<int*>(u8 + l.tickets);
    a.part = reinterpret_cast<float*>(u8 + l.part);
    // The product may start while the kernel right ahead of it, which fills
    // the token tiles, runs: it waits for it before it reads one, and
    // everything before that kernel has ended by then.
    return cuda_status(launch_mx4_gemm(a, dev.sms, true, st));
}

}  // extern "C"
