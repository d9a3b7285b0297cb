// Host launchers of the operators that take any number of tokens (routing,
// the sort by expert, row movement, MXFP4).  moeq_rows_api.cu validates the
// arguments of the C ABI and calls these.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moeq.h"
#include "moeq_once.h"

namespace moeq {

// Raises a kernel's dynamic shared memory limit to `bytes` on the current
// device (`once`: the kernel's own static).  The call costs about a
// microsecond, a small launch's half.
cudaError_t raise_smem(OncePerDevice& once, const void* kernel, int bytes);

// A launch that may be scheduled while the kernel ahead on the stream still
// runs (programmatic dependent launch).  Kernels launched so begin with
// chain(), which waits for everything ahead before any access to memory and
// only then lets the next such launch be scheduled: the order of a stream,
// without the launch latency between its kernels.
//
// Such a kernel is resident while its inputs are still being written, so it
// reads them with plain loads.  A non-coherent one (__ldg, or what the
// compiler makes of a load through a `const T* __restrict__` parameter) is
// for memory that nobody writes while the kernel runs, and the compiler may
// move it ahead of chain().
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void chain() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// A matrix of rows: base, leading dimension in elements, element type.
struct RowsIn {
    const void* p;
    int64_t ld;
    int f32;
};
struct RowsOut {
    void* p;
    int64_t ld;
    int f32;
};

cudaError_t launch_route_rows(const float* logits, int64_t ld, int T, int E, int k, int32_t* id, float* w,
                              cudaStream_t stream);
cudaError_t launch_route_rows_grad(const float* dw, const int32_t* id, const float* w, int T, int E, int k,
                                   float* dlogits, int64_t ld, cudaStream_t stream);
cudaError_t launch_expert_sort(const int32_t* id, int T, int k, int E, int32_t* offs, int32_t* pair_row,
                               int32_t* row_pair, cudaStream_t stream);
cudaError_t launch_gather_rows(RowsIn x, int T, int H, int k, const int32_t* offs, int E, const int32_t* pair_row,
                               RowsOut xs, cudaStream_t stream);
// out[t] = base[t] + sum_j w[t, j] * y[pair_row[t, j]]; w == NULL: weights 1.
cudaError_t launch_combine_rows(RowsIn y, int T, int H, int k, const int32_t* pair_row, const float* w, RowsIn base,
                                RowsOut out, cudaStream_t stream);
cudaError_t launch_combine_rows_grad(RowsIn dout, RowsIn y, int T, int H, int k, const int32_t* offs, int E,
                                     const int32_t* pair_row, const float* w, RowsOut dy, float* dw,
                                     cudaStream_t stream);

// ------------------------------------------------------------------ MXFP4
// Weights are tile-major: tile (e, nb, kb) is the 128 x 256 block of rows
// nb*128.. and columns kb*256.. of expert e: 16 KiB of codes (rows of 128
// bytes, the 16-byte chunk c of row r stored at chunk c ^ (r % 8)) and 1 KiB
// of scales: per 128 columns 512 bytes, the word of row r (its four scale
// bytes, lowest column first) at word (r % 32) * 4 + r / 32.  Rows and
// columns past N and K are zero.
constexpr int kMx4TileRows = 128, kMx4TileCols = 256, kMx4TileBytes = 16384, kMx4TileScaleBytes = 1024;

// Activations: codes [rows, K/2], scales [rows, pitch] bytes (eight for every
// 256 columns; those past K are zero).
__host__ __device__ constexpr int mx4_scale_pitch(int K) { return (K + kMx4TileCols - 1) / kMx4TileCols * 8; }
__host__ __device__ constexpr int mx4_kb(int K) { return (K + kMx4TileCols - 1) / kMx4TileCols; }
__host__ __device__ constexpr int mx4_nb(int N) { return (N + kMx4TileRows - 1) / kMx4TileRows; }

// act: x is [rows, 2K] and silu(x[:, :K]) * x[:, K:] is quantised.
cudaError_t launch_mx4_quant_act(RowsIn x, int rows, int K, int act, uint8_t* codes, uint8_t* scales,
                                 int sms, cudaStream_t stream);
cudaError_t launch_mx4_dequant_act(const uint8_t* codes, const uint8_t* scales, int rows, int K, RowsOut out,
                                   cudaStream_t stream);
cudaError_t launch_mx4_quant_weight(const void* w, int w_f32, int E, int N, int K, uint8_t* tiles, uint8_t* stiles,
                                    cudaStream_t stream);
cudaError_t launch_mx4_pack_weight(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, uint8_t* tiles,
                                   uint8_t* stiles, cudaStream_t stream);

// A product's rows, quantised and laid out in token tiles as the tensor core
// reads them: tile g of expert e holds up to nt of its rows; K block kb of it
// is nt rows of 128 bytes at ((g * KB + kb) * nt) * 128 (chunks rotated as in
// a weight tile), its scales mx4_tile_scale_bytes(nt) at (g * KB + kb) times
// that (a weight tile's order, one more 512 bytes for rows 128..).
constexpr int kMx4Tickets = 1024;  // units that are cut (a quarter of the SMs at most)
__host__ __device__ constexpr int mx4_tile_scale_bytes(int nt) { return nt > 128 ? 2048 : 1024; }
// Most rows of one token tile for R rows over E experts, and what tiles' rows
// are rounded to: 16, or 32 where pairs of CTAs multiply them.
struct Mx4Tiling {
    int nt, align;
};
Mx4Tiling mx4_tiling(int R, int E);
// Most token tiles there can be.
__host__ __device__ constexpr int64_t mx4_max_tiles(int R, int E, int nt) { return R / nt + (E < R ? E : R); }

// Which activation row each row reads, and where it lies.
struct Mx4Plan {
    const int32_t* offs;      // [E + 1]
    const int32_t* row_pair;  // [R] or NULL: row r reads activation row r
    int E, R, top_k, rows;    // rows: activation rows
    int nt, align;
};

// Source of the tiles: a matrix to quantise (act as in
// launch_mx4_quant_act), or codes and scales made beforehand.
struct Mx4Source {
    RowsIn x;
    int act;
    const uint8_t* codes;     // NULL: x is quantised
    const uint8_t* scales;
};
cudaError_t launch_mx4_act_tiles(const Mx4Source& src, const Mx4Plan& plan, int K, uint8_t* tiles, uint8_t* stiles,
                                 int sms, cudaStream_t stream);

struct Mx4GemmArgs {
    const uint8_t* w;       // weight tiles and their scales
    const uint8_t* sw;
    const uint8_t* a;       // token tiles and their scales
    const uint8_t* sa;
    Mx4Plan plan;
    void* y;
    int64_t ld_y;
    int y_f32;
    int K, N;
    int stages;
    int* tickets;           // kMx4Tickets, zero between launches
    float* part;            // grid slots of nt * 128 floats
    int* status;
};
// pdl: start while the kernel ahead on the stream (which writes the token
// tiles, and nothing else of the arguments) runs.
cudaError_t launch_mx4_gemm(Mx4GemmArgs a, int grid, bool pdl, cudaStream_t stream);

}  // namespace moeq
