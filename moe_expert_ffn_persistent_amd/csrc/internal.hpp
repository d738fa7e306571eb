// Internal declarations shared by the host API and the kernel launchers of
// the persistent MoE expert-FFN library. Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "moe_ffn.h"

namespace moe {

// Arguments of the layout kernels.
struct LayoutArgs {
  int N, E, k, e0, L, block_m;
  const float* logits;     // [N, E] or nullptr
  const float* bias;       // [E] or nullptr
  int32_t* topk_idx;       // [N, k]
  float* topk_w;           // [N, k]
  int32_t* counts;         // [L]
  int32_t* row_offset;     // [L+1]
  int32_t* tile_offset;    // [L+1]
  int32_t* row_pair;       // [N*k]
  float* row_weight;       // [N*k]
  int32_t* pair_row;       // [N*k]
  int32_t* totals;         // [4]
  int32_t* block_counts;   // [nchunks, L]
  int nchunks;
};

constexpr int kLayoutChunk = 256;    // flat pairs per layout workgroup
constexpr int kTraceWords = MOE_TRACE_WORDS;   // uint32 words per task record

hipError_t launch_layout(const LayoutArgs& a, hipStream_t stream);

// Store burst-gap probe (burst.hip).
struct BurstArgs {
  char* dst;                // destination buffer
  size_t dst_bytes;
  uint32_t* stamps;         // [producers][bursts][2] wall clock: issue start, issue end
  int producers;            // K workgroups
  int bytes_per_burst;      // B per producer, multiple of 4096 and of row_bytes
  int bursts;
  int row_bytes;            // contiguous bytes per destination row, multiple of 16
  int control;              // 1: rows confined to a 256 KiB region (stays in L2)
  long long gap_ticks;      // wall-clock ticks of idling after each burst
};

hipError_t launch_burst(const BurstArgs& a, hipStream_t stream);

// MFMA issue-rate probe (mfma_probe.hip)
size_t mfma_probe_operand_bytes();
int mfma_probe_threads();
hipError_t launch_mfma_probe(int format, int blocks, long long iters, const void* ops, long long* stamps,
                             float* sink, hipStream_t stream);

// Arguments of the persistent FFN kernel. Passed by value; the slice tables
// are copied to LDS at kernel start.
struct FfnArgs {
  int S, T, k, L, H, I;
  int N1, N2;              // Linear-1 / Linear-2 N-tiles per scheduler row
  int grid;                // persistent workgroups (== gridDim.x)
  int xcd_group;           // logical-id placement: 0 = consecutive ids per XCD; R > 0 = grouped by
                           // Linear-1 N-tile (N1 == 8R, N1 | grid): see logical_instance
  int xcd_bx;              // with xcd_group: XCD blocks along the N-tiles (1, 2, 4 or 8)
  int schedule;            // moe_schedule
  int lead_d;              // Interleaved lead D (>= 1)
  int experts_per_wave;    // 0 = greedy
  int debug_skip_row;      // -1 = off
  int trace_cap;
  long long timeout_ticks; // wall-clock ticks before a wait gives up
  const void* x[MOE_MAX_SLICES];
  const float* xs[MOE_MAX_SLICES];   // fp8: fp32 1x128 scales; W4A8: E8M0 bytes per 1x32
  void* comb[MOE_MAX_SLICES];
  const void* w1;
  const float* w1s;        // fp8: fp32 128x128 scales; W4A8: E8M0 bytes per 1x32
  const void* w2;
  const float* w2s;
  const int32_t* row_offset;
  const int32_t* tile_offset;
  const int32_t* row_pair;
  const float* row_weight;
  void* h;                 // [P_cap * block_m, I] intermediate activations
  float* hs;               // fp8: [P_cap * block_m, I/128] fp32 scales; W4A8:
                           // [P_cap * block_m, I/32] E8M0 bytes
  int32_t* l2_full;        // [P_cap] finished Linear-1 tiles per row
  int32_t* done;           // [1] finished workgroups
  int32_t* status;         // device status word or nullptr
  uint32_t* trace;         // task trace or nullptr
};

// Tile configurations. Each id maps to one kernel instantiation.
struct TileInfo {
  int id;
  int dtype;       // moe_dtype
  int block_m;     // tokens per M-block
  int block_n;     // features per N-tile (both GEMMs)
  int threads;
};


struct CheckArgs {
  int S, T, k, H, L;
  void* comb[MOE_MAX_SLICES];
  const int32_t* pair_row;
  void* y;
  int y_bf16;              // y is bf16 (round to nearest even) instead of fp32
  const int32_t* status;   // FFN status word or nullptr (copied to report[3])
  int32_t* report;
};
hipError_t launch_check(const CheckArgs& a, hipStream_t stream);

// Operators around the FFN (rows.hip, swiglu.hip, gemm_any.hip, ...). Leading
// dimensions of rows are in bytes for RowsArgs, in elements elsewhere.
struct RowsArgs {
  const void* in;
  void* out;
  const int32_t* index;        // row_pair (dispatch) or pair_row (combine)
  const int32_t* row_offset;   // dispatch
  long long rows, pairs;       // capacity; tokens * k
  long long ld_in, ld_out;
  int k, hidden, elem, L;
};
hipError_t launch_dispatch_rows(const RowsArgs& a, hipStream_t s);
// weights: fp32 of every pair, or nullptr (1)
hipError_t launch_combine_rows(const RowsArgs& a, const float* weights, bool bf16_out, hipStream_t s);

struct CombineBackwardArgs {
  const void *dy, *rows;
  const int32_t* pair_row;
  const float* weights;
  void* drows;
  float* dweights;
  long long cap, ld_dy, ld_rows, ld_drows;   // rows that the buffers hold; strides in elements
  int tokens, k, hidden;
  bool dy_fp32;
};
hipError_t launch_combine_backward(const CombineBackwardArgs& a, hipStream_t s);

// RMS norm (norm.hip), strides in elements (codes and scale bytes in bytes).
// Forward: stream = x + residual (x without one), out = stream / rms * weight in
// the format; backward: out (of dy) and dx of the stream, partial sums of dweight.
struct NormArgs {
  const void *x, *residual, *weight, *dy;
  void *out, *scales, *stream, *dx;   // stream: where the sum is stored
  const void* dresidual;
  float *dweight, *part;              // part: [groups, hidden], or dweight itself
  long long rows, ld_x, ld_residual, ld_stream, ld_out, ld_scales, ld_dy, ld_dresidual, ld_dx;
  int hidden, format;                 // MOE_NORM_*; backward: of dy
  float eps;
  bool fp32, weight_fp32;             // type of the stream (x, residual, dx, ...); of weight
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);
// workgroups of the backward pass, each with a partial sum of dweight
int norm_backward_groups(long long rows, int hidden, bool fp32);
hipError_t launch_rms_norm_backward(const NormArgs& a, hipStream_t s);

struct SwigluArgs {
  const void *a, *dh;
  const float* weight;
  const int32_t* row_offset;   // nullptr: every row
  void *h, *da;
  float *scales, *dweight;
  long long rows, ld_a, ld_h, ld_scales, ld_da;
  int inter, L;
  bool vec;                    // rows are 16-byte aligned (codes: 8-byte)
};
hipError_t launch_swiglu(const SwigluArgs& a, bool fp8, hipStream_t s);
hipError_t launch_swiglu_backward(const SwigluArgs& a, hipStream_t s);

struct QuantArgs {
  const void* x;
  const int32_t* row_offset;
  void* codes;
  float* scales;
  long long rows, ld_x, ld_codes, bs_x, bs_codes;
  int batch, cols, L;
  bool vec, vec16;             // rows of x 16-byte, of codes 8-byte and 16-byte aligned
};
hipError_t launch_quantize(const QuantArgs& a, int block_rows, bool fp32, hipStream_t s);

// Microscaled formats (mx_quantize.hip); strides of codes and scales in bytes
struct MxQuantArgs {
  const void* x;
  const int32_t* row_offset;
  uint8_t *codes, *scales;
  long long rows, ld_x, ld_codes, ld_scales, bs_x, bs_codes, bs_scales;
  int batch, cols, L;
};
hipError_t launch_quantize_mx(const MxQuantArgs& a, bool e2m1, bool fp32, hipStream_t s);

// Grouped products: x [rows, k], w [L, n, k], y [rows, n], one of them written
// (op: MOE_GROUPED_*); the block-scaled e4m3 product is the forward form with
// scales. row_offset nullptr: one expert with every row.
struct GemmArgs {
  const int32_t* row_offset;
  void *x, *w, *y;
  const float *xs, *ws;
  long long ld_x, ld_w, ld_y, es_w, ld_xs;
  int op, L, rows, n, k;
  bool out_bf16, accumulate;
  int expected;                // rows expected in all experts together
  // The sum cut into `splits` ranges of whole stages (1: not cut): range s adds
  // up in fp32 at s * part elements past the output
  int splits;
  long long part;
  // The product of MX operands: xs and ws are E8M0 bytes, all strides but ld_y's in bytes
  long long ld_ws, es_ws;
  bool x_e2m1, vec_out;        // rows of y are 16-byte aligned
};
constexpr int kCus = 256;   // compute units, places for a persistent workgroup
hipError_t launch_gemm_any(const GemmArgs& a, bool fp8, hipStream_t s);
// tiles 1 .. kBf16GemmTiles (kFp8GemmTiles) of the 16-byte kernels
constexpr int kBf16GemmTiles = 9, kFp8GemmTiles = 9;
struct GemmTile {
  int tm, tn, occ, kw;   // rows, columns, workgroups per compute unit, wavefronts that split the sum
  double a, c, b, o;     // us: a stage alone, with a workgroup on every compute unit, with occ of them, a tile's ends
  bool once;             // only for calls that give no compute unit a second tile
};
extern const GemmTile kBf16GemmTileTable[], kDgradTiles[], kWgradTiles[], kFp8GemmTileTable[];   // id - 1
// Most output tiles of tm x tn that a call has, over all ranges of its sum. The tile
// kernels count them in int, and the kernels of any size, which take over from
// kMostTiles on, add up no ranges.
constexpr long long kMostTiles = 1ll << 30;
inline long long gemm_tiles(const GemmArgs& a, int tm, int tn) {
  const long long nj = ((a.op == MOE_GROUPED_FORWARD ? a.n : a.k) + tn - 1) / tn;
  const long long mi = a.op == MOE_GROUPED_WGRAD ? (long long)a.L * ((a.n + tm - 1) / tm) : (a.rows + (long long)a.L * (tm - 1)) / tm;
  return nj * mi * a.splits;
}
// The same call with its sum cut into a.splits ranges, written to `ws` (fp32, one
// output's elements a range), and the joining of them into a's output
GemmArgs split_args(const GemmArgs& a, float* ws);
hipError_t launch_join_splits(const GemmArgs& a, const float* ws, hipStream_t s);
hipError_t launch_gemm_bf16(int id, const GemmArgs& a, hipStream_t s);
hipError_t launch_gemm_fp8(int id, const GemmArgs& a, hipStream_t s);
constexpr int kMxGemmTiles = 10;
extern const GemmTile kMxTiles[2][kMxGemmTiles];   // by the type of x: e4m3, e2m1; id - 1; tm 0: not a tile of it
hipError_t launch_gemm_mx(int id, const GemmArgs& a, hipStream_t s);
hipError_t launch_gemm_mx_any(const GemmArgs& a, hipStream_t s);

hipError_t launch_zero(void* p, size_t bytes, hipStream_t stream);

// The shape checks every entry point makes (api.cpp).
bool shape_valid(const moe_shape* s);

}  // namespace moe
