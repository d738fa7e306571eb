// Host side of the operators around the expert FFN: argument checks and
// kernel choice. Nothing here allocates, waits or keeps state.
#include <hip/hip_runtime.h>

#include <cmath>

#include "internal.hpp"

using namespace moe;

namespace {

constexpr long long kMaxRows = 1ll << 28;
constexpr int kMaxCols = 1 << 20;
// elements between rows or matrices: the checks below multiply by up to
// kMaxRows, the kernels' byte offsets stay inside 64 bits
constexpr long long kMaxStride = 1ll << 32, kMaxMatrix = 1ll << 52;
// tokens: dispatch only multiplies by them; combine has a workgroup of 256
// threads for a token at most, and fewer than 2^32 threads a launch
constexpr long long kMaxTokens = 1ll << 40, kMaxCombineTokens = 1ll << 23;

int32_t done(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// offsets, indices, fp32 scales and weights
template <class... P>
bool words(const P*... p) { return (aligned(p, 4) && ...); }

// a row stride of rows of `cols` elements
bool stride_ok(long long ld, long long cols) { return ld >= cols && ld <= kMaxStride; }

// the distance between `count` matrices of `rows` such rows
bool matrix_stride_ok(long long stride, long long count, long long rows, long long ld, long long cols) {
  return count <= 1 || (stride >= (rows - 1) * ld + cols && stride <= kMaxMatrix);
}

bool dtype_ok(int32_t d) { return d == MOE_Y_FP32 || d == MOE_Y_BF16; }

int expected_rows(int64_t expected, int64_t rows) {
  return (int)(expected > 0 && expected < rows ? expected : rows);
}

// M-blocks of tm rows that the experts are expected to need: a partial block
// each on top of their even share, one for an expert with few rows, none for
// an expert that no row reaches.
double expected_blocks(double rows, int L, int tm) {
  if (L == 1) return std::ceil(rows / tm);
  const double avg = rows / L;
  return L * std::max(1.0 - std::exp(-avg), avg / tm + 0.5);
}

// Predicted microseconds of a call in tile t: every compute unit works through
// its share of the tiles one after the other, `stages` stages and a fixed cost
// each. A stage's time grows from the tile's when few compute units work (a) to
// that with all of them at work (c: clock, L2 and memory are shared then); with
// two workgroups on a compute unit a stage of one of them takes 2 b.
// Fitted to calls of 1 to 16384 rows, 1 to 128 experts and 80 to 28672 features,
// each timed with every tile: over 88 calls of each product the tile chosen took
// 1.8% (forward), 2.3% (dgrad), 0.9% (wgrad) and 1.6% (e4m3) longer than the best
// one in the mean, 45% at worst (wgrad of 256 rows; a few rows to many experts).
double predicted(const GemmTile& t, double tiles, double stages) {
  const double q = std::max(1.0, std::ceil(tiles / kCus - 0.02));
  const double one = t.a + (t.c - t.a) * std::min(1.0, tiles / kCus);
  if (t.occ == 1) return q * (stages * one + t.o);
  const double pairs = std::floor(q / 2);
  return pairs * (stages * std::max(one, 2 * t.b) + t.o) + (q - 2 * pairs) * (stages * one + t.o);
}

constexpr double kJoinUs = 3, kJoinRate = 5e6, kReadRate = 5.5e6;   // bytes a us

struct Choice {
  int tile, splits;
};

// Tile (or the one asked for) and ranges of the sum, up to what `room` fp32
// elements of workspace hold. Joining costs a launch and a pass over the ranges,
// and ranges cannot be added up faster than the operands are read. Over 160 calls
// of 1 to 16384 rows, 1 to 32 experts and 72 to 7168 features, each timed with
// every tile and 1 to 16 ranges, the choice took 2.5% longer than the best one in
// the mean, 34% at worst; without ranges some took 2 to 5 times as long (weight
// gradient 256 x 128 of 16000 rows 79 us, in 16 ranges 16).
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
constexpr int kMaxSplits = 64;
constexpr long long kMaxWorkspace = 256ll << 20;

Choice choose(const GemmTile* tiles, int n, const GemmArgs& a, int bk, int tile, int splits, long long room) {
  const bool wgrad = a.op == MOE_GROUPED_WGRAD;
  const int nj = a.op == MOE_GROUPED_FORWARD ? a.n : a.k, nc = a.op == MOE_GROUPED_FORWARD ? a.k : a.n;
  const long long part = split_args(a, nullptr).part;
  const double written = wgrad ? (double)part : (double)a.expected * nj;
  const double touched = std::min<double>(a.L, a.expected) * a.n * a.k, rows = (double)a.expected * ((double)a.n + a.k);
  const double read = (touched + rows) * (bk == 128 ? 1 : 2) / kReadRate;
  Choice best{tile > 0 ? tile : 1, splits > 0 ? splits : 1};
  double least = 1e300;
  for (int i = tile > 0 ? tile - 1 : 0; i < (tile > 0 ? tile : n); ++i) {
    const GemmTile& t = tiles[i];
    if (t.tm == 0) continue;   // not a tile of this product
    const double blocks = wgrad ? (double)a.L * ((a.n + t.tm - 1) / t.tm) : expected_blocks(a.expected, a.L, t.tm);
    const double stages = wgrad ? (double)a.expected / a.L / bk + 0.5 : std::max(1.0, (double)nc / bk / t.kw);
    for (const int candidate : kSplits) {
      const int s = splits > 0 ? splits : candidate;
      if (splits == 0 && s > 1 && (s * part > room || stages < 4 * s)) continue;
      const double count = s * blocks * ((nj + t.tn - 1) / t.tn);
      if (t.once && count > kCus && tile == 0) continue;
      const double us = s == 1 ? predicted(t, count, stages)
                               : std::max(predicted(t, count, std::ceil(stages / s)), read) + kJoinUs + s * written * 8 / kJoinRate;
      if (us < least) {
        least = us;
        best = Choice{i + 1, s};
      }
    }
  }
  return best;
}

// the ranges and workspace of a *_split call
bool split_ok(int32_t splits, int64_t bytes) { return splits >= 0 && splits <= kMaxSplits && bytes >= 0; }

// One product: whole, or in ranges joined afterwards
template <class Launch>
int32_t run(const GemmArgs& a, Choice c, float* ws, hipStream_t s, Launch launch) {
  if (c.splits == 1) return done(launch(c.tile, a, s));
  GemmArgs b = a;
  b.splits = c.splits;
  const hipError_t e = launch(c.tile, split_args(b, ws), s);
  return e != hipSuccess ? done(e) : done(launch_join_splits(b, ws, s));
}

// Bytes that the automatic choice of a call takes
int64_t workspace_of(const GemmTile* tiles, int n, const GemmArgs& a, int bk, int tile, int splits) {
  const Choice c = choose(tiles, n, a, bk, tile, splits, kMaxWorkspace / 4);
  return c.splits > 1 ? c.splits * split_args(a, nullptr).part * 4 : 0;
}

bool grouped_ok(const moe_grouped_params* p) {
  return p && p->op >= MOE_GROUPED_FORWARD && p->op <= MOE_GROUPED_WGRAD && p->num_experts >= 1 &&
         p->num_experts <= MOE_MAX_LOCAL_EXPERTS && p->rows >= 0 && p->rows <= kMaxRows && p->expected_rows >= 0 &&
         p->n >= 1 && p->n <= kMaxCols && p->k >= 1 && p->k <= kMaxCols && stride_ok(p->ld_x, p->k) &&
         stride_ok(p->ld_w, p->k) && stride_ok(p->ld_y, p->n) &&
         matrix_stride_ok(p->expert_stride_w, p->num_experts, p->n, p->ld_w, p->k) && dtype_ok(p->out_dtype) &&
         p->tile >= 0 && (!p->accumulate || p->op == MOE_GROUPED_WGRAD);
}

// The 16-byte kernels' sizes: rows of every operand start and end on 16 bytes,
// and their lane offsets (256 rows of a tile) fit 32 bits.
bool grouped_fast(const moe_grouped_params* p) {
  return p->n % 8 == 0 && p->k % 8 == 0 && p->ld_x % 8 == 0 && p->ld_w % 8 == 0 && p->ld_y % 8 == 0 &&
         p->expert_stride_w % 8 == 0 && std::max(p->ld_x, std::max(p->ld_w, p->ld_y)) <= (1 << 22);
}

const GemmTile* grouped_tiles(const moe_grouped_params* p) {
  return p->op == MOE_GROUPED_WGRAD ? kWgradTiles : p->op == MOE_GROUPED_DGRAD ? kDgradTiles : kBf16GemmTileTable;
}

// an id the call's sizes can take
bool grouped_tile_ok(const moe_grouped_params* p) {
  return p->tile == 0 || (p->tile <= kBf16GemmTiles && grouped_tiles(p)[p->tile - 1].tm > 0);
}

GemmArgs grouped_args(const moe_grouped_params* p) {
  GemmArgs a{};
  a.ld_x = p->ld_x;
  a.ld_w = p->ld_w;
  a.ld_y = p->ld_y;
  a.es_w = p->expert_stride_w;
  a.op = p->op;
  a.L = p->num_experts;
  a.rows = (int)p->rows;
  a.n = p->n;
  a.k = p->k;
  a.out_bf16 = p->out_dtype == MOE_Y_BF16;
  a.accumulate = p->accumulate != 0;
  a.expected = expected_rows(p->expected_rows, p->rows);
  a.splits = 1;
  return a;
}

int32_t grouped(const moe_grouped_params* p, const int32_t* row_offset, void* x, void* w, void* y, int splits,
                void* workspace, int64_t bytes, hipStream_t stream) {
  const bool wgrad = p->op == MOE_GROUPED_WGRAD, fwd = p->op == MOE_GROUPED_FORWARD;
  if (p->rows == 0 && (!wgrad || p->accumulate)) return MOE_OK;
  if (!row_offset || !w || (p->rows && (!x || !y)) || !words(row_offset)) return MOE_ERR_INVALID_ARG;
  const size_t oe = p->out_dtype == MOE_Y_BF16 ? 2 : 4;
  if (!aligned(x, !fwd && !wgrad ? oe : 2) || !aligned(y, fwd ? oe : 2) || !aligned(w, wgrad ? oe : 2) ||
      !aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  GemmArgs a = grouped_args(p);
  a.row_offset = row_offset;
  a.x = x;
  a.w = w;
  a.y = y;
  const bool fast = grouped_fast(p) && aligned(x, 16) && aligned(w, 16) && aligned(y, 16);
  if (!grouped_tile_ok(p) || (p->tile > 0 && !fast)) return MOE_ERR_UNSUPPORTED;
  if (!fast) return done(launch_gemm_any(a, false, stream));
  const long long room = workspace ? bytes / 4 : 0;
  if (splits > 1 && splits * split_args(a, nullptr).part > room) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return run(a, choose(grouped_tiles(p), kBf16GemmTiles, a, 64, p->tile, splits, room), static_cast<float*>(workspace),
             stream, launch_gemm_bf16);
}

bool fp8_ok(const moe_fp8_params* p) {
  return p && p->num_experts >= 1 && p->num_experts <= MOE_MAX_LOCAL_EXPERTS && p->rows >= 0 && p->rows <= kMaxRows &&
         p->expected_rows >= 0 && p->n >= 1 && p->n <= kMaxCols && p->k >= 1 && p->k <= kMaxCols &&
         stride_ok(p->ld_x, p->k) && stride_ok(p->ld_w, p->k) && stride_ok(p->ld_y, p->n) &&
         stride_ok(p->ld_xs, (p->k + 127) / 128) &&
         matrix_stride_ok(p->expert_stride_w, p->num_experts, p->n, p->ld_w, p->k) && dtype_ok(p->out_dtype) &&
         p->tile >= 0;
}

bool fp8_fast(const moe_fp8_params* p) {
  return p->n % 8 == 0 && p->k % 16 == 0 && p->ld_x % 16 == 0 && p->ld_w % 16 == 0 && p->ld_y % 8 == 0 &&
         p->expert_stride_w % 16 == 0 && std::max(p->ld_x, std::max(p->ld_w, p->ld_xs)) <= (1 << 22);
}

GemmArgs fp8_args(const moe_fp8_params* p) {
  GemmArgs a{};
  a.ld_x = p->ld_x;
  a.ld_w = p->ld_w;
  a.ld_y = p->ld_y;
  a.es_w = p->expert_stride_w;
  a.ld_xs = p->ld_xs;
  a.op = MOE_GROUPED_FORWARD;
  a.L = p->num_experts;
  a.rows = (int)p->rows;
  a.n = p->n;
  a.k = p->k;
  a.out_bf16 = p->out_dtype == MOE_Y_BF16;
  a.expected = expected_rows(p->expected_rows, p->rows);
  a.splits = 1;
  return a;
}

int32_t fp8(const moe_fp8_params* p, const int32_t* row_offset, const void* x, const float* x_scales, const void* w,
            const float* w_scales, void* y, int splits, void* workspace, int64_t bytes, hipStream_t stream) {
  if (!row_offset && p->num_experts != 1) return MOE_ERR_INVALID_ARG;
  if (p->rows == 0) return MOE_OK;
  if (!x || !x_scales || !w || !w_scales || !y || !aligned(y, p->out_dtype == MOE_Y_BF16 ? 2 : 4) || !aligned(workspace, 16) ||
      !words(row_offset, x_scales, w_scales))
    return MOE_ERR_INVALID_ARG;
  GemmArgs a = fp8_args(p);
  a.row_offset = row_offset;
  a.x = const_cast<void*>(x);
  a.w = const_cast<void*>(w);
  a.y = y;
  a.xs = x_scales;
  a.ws = w_scales;
  const bool fast = fp8_fast(p) && aligned(x, 16) && aligned(w, 16) && aligned(y, 16);
  if (p->tile > kFp8GemmTiles || (p->tile > 0 && !fast)) return MOE_ERR_UNSUPPORTED;
  if (!fast) return done(launch_gemm_any(a, true, stream));
  const long long room = workspace ? bytes / 4 : 0;
  if (splits > 1 && splits * split_args(a, nullptr).part > room) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return run(a, choose(kFp8GemmTileTable, kFp8GemmTiles, a, 128, p->tile, splits, room), static_cast<float*>(workspace),
             stream, launch_gemm_fp8);
}

}  // namespace

extern "C" {

int32_t moe_dispatch_rows(const moe_rows_params* p, const void* x, const int32_t* row_pair,
                          const int32_t* row_offset, void* out, void* stream) {
  if (!p || p->tokens < 0 || p->rows < 0 || p->rows > kMaxRows || p->top_k < 1 || p->top_k > 16 || p->hidden < 1 ||
      p->hidden > kMaxCols || (p->elem_bytes != 1 && p->elem_bytes != 2 && p->elem_bytes != 4) ||
      p->num_experts < 1 || p->num_experts > MOE_MAX_LOCAL_EXPERTS || !stride_ok(p->ld_tokens, p->hidden) ||
      !stride_ok(p->ld_rows, p->hidden) || p->tokens > kMaxTokens)
    return MOE_ERR_INVALID_ARG;
  if (p->rows == 0) return MOE_OK;
  if (!row_pair || !row_offset || !out || (p->tokens && !x) || !words(row_pair, row_offset)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, p->elem_bytes) || !aligned(out, p->elem_bytes)) return MOE_ERR_INVALID_ARG;
  RowsArgs a{};
  a.in = x;
  a.out = out;
  a.index = row_pair;
  a.row_offset = row_offset;
  a.rows = p->rows;
  a.pairs = p->tokens * p->top_k;
  a.ld_in = p->ld_tokens * p->elem_bytes;
  a.ld_out = p->ld_rows * p->elem_bytes;
  a.k = p->top_k;
  a.hidden = p->hidden;
  a.elem = p->elem_bytes;
  a.L = p->num_experts;
  return done(launch_dispatch_rows(a, (hipStream_t)stream));
}

int32_t moe_combine_rows(const moe_rows_params* p, const void* in, const int32_t* pair_row, void* y, void* stream) {
  if (!p || p->tokens < 0 || p->rows < 0 || p->rows > kMaxRows || p->top_k < 1 || p->top_k > 16 || p->hidden < 1 ||
      p->hidden > kMaxCols || p->elem_bytes != 2 || !dtype_ok(p->out_dtype) || !stride_ok(p->ld_tokens, p->hidden) ||
      !stride_ok(p->ld_rows, p->hidden) || p->tokens > kMaxCombineTokens)
    return MOE_ERR_INVALID_ARG;
  if (p->tokens == 0) return MOE_OK;
  if (!pair_row || !y || (p->rows && !in) || !words(pair_row)) return MOE_ERR_INVALID_ARG;
  const size_t out_elem = p->out_dtype == MOE_Y_BF16 ? 2 : 4;
  if (!aligned(in, 2) || !aligned(y, out_elem)) return MOE_ERR_INVALID_ARG;
  RowsArgs a{};
  a.in = in;
  a.out = y;
  a.index = pair_row;
  a.rows = p->rows;
  a.pairs = p->tokens * p->top_k;
  a.ld_in = p->ld_rows * 2;
  a.ld_out = p->ld_tokens * (long long)out_elem;
  a.k = p->top_k;
  a.hidden = p->hidden;
  a.elem = 2;
  return done(launch_combine_rows(a, p->out_dtype == MOE_Y_BF16, (hipStream_t)stream));
}

int32_t moe_grouped_matmul(const moe_grouped_params* p, const int32_t* row_offset, void* x, void* w, void* y,
                           void* stream) {
  if (!grouped_ok(p)) return MOE_ERR_INVALID_ARG;
  return grouped(p, row_offset, x, w, y, 1, nullptr, 0, (hipStream_t)stream);
}

int32_t moe_grouped_matmul_split(const moe_grouped_params* p, const int32_t* row_offset, void* x, void* w, void* y,
                                 void* workspace, void* stream) {
  if (!grouped_ok(p) || !split_ok(p->splits, p->workspace_bytes)) return MOE_ERR_INVALID_ARG;
  return grouped(p, row_offset, x, w, y, p->splits, workspace, p->workspace_bytes, (hipStream_t)stream);
}

int64_t moe_grouped_workspace_bytes(const moe_grouped_params* p) {
  if (!grouped_ok(p) || !split_ok(p->splits, 0) || !grouped_fast(p) || !grouped_tile_ok(p)) return 0;
  return workspace_of(grouped_tiles(p), kBf16GemmTiles, grouped_args(p), 64, p->tile, p->splits);
}

int32_t moe_swiglu(const moe_swiglu_params* p, const void* a_, const float* row_weight, const int32_t* row_offset,
                   void* h, float* h_scales, void* stream) {
  if (!p || p->rows < 0 || p->rows > kMaxRows || p->inter < 1 || p->inter > kMaxCols ||
      !stride_ok(p->ld_a, 2ll * p->inter) || !stride_ok(p->ld_h, p->inter) || (p->out_format != MOE_SWIGLU_BF16 && p->out_format != MOE_SWIGLU_FP8) ||
      (row_offset && (p->num_experts < 1 || p->num_experts > MOE_MAX_LOCAL_EXPERTS)))
    return MOE_ERR_INVALID_ARG;
  const bool fp8 = p->out_format == MOE_SWIGLU_FP8;
  if (fp8 && !stride_ok(p->ld_scales, (p->inter + 127) / 128)) return MOE_ERR_INVALID_ARG;
  if (p->rows == 0) return MOE_OK;
  if (!a_ || !h || (fp8 && !h_scales) || !aligned(a_, 2) || (!fp8 && !aligned(h, 2)) ||
      !words(row_weight, row_offset, h_scales))
    return MOE_ERR_INVALID_ARG;
  SwigluArgs a{};
  a.a = a_;
  a.weight = row_weight;
  a.row_offset = row_offset;
  a.h = h;
  a.scales = h_scales;
  a.rows = p->rows;
  a.ld_a = p->ld_a;
  a.ld_h = p->ld_h;
  a.ld_scales = p->ld_scales;
  a.inter = p->inter;
  a.L = p->num_experts;
  a.vec = aligned(a_, 16) && aligned(h, fp8 ? 8 : 16) && p->inter % 8 == 0 && p->ld_a % 8 == 0 && p->ld_h % 8 == 0;
  return done(launch_swiglu(a, fp8, (hipStream_t)stream));
}

int32_t moe_swiglu_backward(const moe_swiglu_params* p, const void* a_, const void* dh, const float* row_weight,
                            const int32_t* row_offset, void* da, float* drow_weight, void* stream) {
  if (!p || p->rows < 0 || p->rows > kMaxRows || p->inter < 1 || p->inter > kMaxCols ||
      !stride_ok(p->ld_a, 2ll * p->inter) || !stride_ok(p->ld_da, 2ll * p->inter) || !stride_ok(p->ld_h, p->inter) ||
      (row_offset && (p->num_experts < 1 || p->num_experts > MOE_MAX_LOCAL_EXPERTS)))
    return MOE_ERR_INVALID_ARG;
  if (p->rows == 0) return MOE_OK;
  if (!a_ || !dh || !da || !aligned(a_, 2) || !aligned(dh, 2) || !aligned(da, 2) ||
      !words(row_weight, row_offset, drow_weight))
    return MOE_ERR_INVALID_ARG;
  SwigluArgs a{};
  a.a = a_;
  a.dh = dh;
  a.weight = row_weight;
  a.row_offset = row_offset;
  a.da = da;
  a.dweight = drow_weight;
  a.rows = p->rows;
  a.ld_a = p->ld_a;
  a.ld_h = p->ld_h;
  a.ld_da = p->ld_da;
  a.inter = p->inter;
  a.L = p->num_experts;
  a.vec = aligned(a_, 16) && aligned(dh, 16) && aligned(da, 16) && p->inter % 8 == 0 && p->ld_a % 8 == 0 &&
          p->ld_h % 8 == 0 && p->ld_da % 8 == 0;
  return done(launch_swiglu_backward(a, (hipStream_t)stream));
}

int32_t moe_quantize_fp8(const moe_quantize_params* p, const void* x, const int32_t* row_offset, void* codes,
                         float* scales, void* stream) {
  if (!p || p->rows < 0 || p->rows > kMaxRows || p->batch < 1 || p->batch > 65535 || p->cols < 1 ||
      p->cols > kMaxCols || (p->block_rows != 1 && p->block_rows != 128) || !dtype_ok(p->in_dtype) ||
      !stride_ok(p->ld_x, p->cols) || !stride_ok(p->ld_codes, p->cols))
    return MOE_ERR_INVALID_ARG;
  if (row_offset && (p->batch != 1 || p->block_rows != 1 || p->num_experts < 1 ||
                     p->num_experts > MOE_MAX_LOCAL_EXPERTS))
    return MOE_ERR_INVALID_ARG;
  if (p->rows == 0) return MOE_OK;
  if (!matrix_stride_ok(p->batch_stride_x, p->batch, p->rows, p->ld_x, p->cols) ||
      !matrix_stride_ok(p->batch_stride_codes, p->batch, p->rows, p->ld_codes, p->cols))
    return MOE_ERR_INVALID_ARG;
  // a workgroup of 512 threads a block, and fewer than 2^32 threads a launch
  if (p->block_rows == 128 && ((p->rows + 127) / 128) * ((p->cols + 127) / 128) >= (1ll << 23))
    return MOE_ERR_UNSUPPORTED;
  const bool fp32 = p->in_dtype == MOE_Y_FP32;
  const int xe = fp32 ? 4 : 2;
  if (!x || !codes || !scales || !aligned(x, xe) || !words(row_offset, scales)) return MOE_ERR_INVALID_ARG;
  QuantArgs a{};
  a.x = x;
  a.row_offset = row_offset;
  a.codes = codes;
  a.scales = scales;
  a.rows = p->rows;
  a.ld_x = p->ld_x;
  a.ld_codes = p->ld_codes;
  a.bs_x = p->batch > 1 ? p->batch_stride_x : 0;
  a.bs_codes = p->batch > 1 ? p->batch_stride_codes : 0;
  a.batch = p->batch;
  a.cols = p->cols;
  a.L = p->num_experts;
  a.vec = aligned(x, 16) && aligned(codes, 8) && (a.ld_x * xe) % 16 == 0 && (a.bs_x * xe) % 16 == 0 &&
          a.ld_codes % 8 == 0 && a.bs_codes % 8 == 0;
  a.vec16 = a.vec && aligned(codes, 16) && a.ld_codes % 16 == 0 && a.bs_codes % 16 == 0;
  return done(launch_quantize(a, p->block_rows, fp32, (hipStream_t)stream));
}

int32_t moe_fp8_matmul(const moe_fp8_params* p, const int32_t* row_offset, const void* x, const float* x_scales,
                       const void* w, const float* w_scales, void* y, void* stream) {
  if (!fp8_ok(p)) return MOE_ERR_INVALID_ARG;
  return fp8(p, row_offset, x, x_scales, w, w_scales, y, 1, nullptr, 0, (hipStream_t)stream);
}

int32_t moe_fp8_matmul_split(const moe_fp8_params* p, const int32_t* row_offset, const void* x, const float* x_scales,
                             const void* w, const float* w_scales, void* y, void* workspace, void* stream) {
  if (!fp8_ok(p) || !split_ok(p->splits, p->workspace_bytes)) return MOE_ERR_INVALID_ARG;
  return fp8(p, row_offset, x, x_scales, w, w_scales, y, p->splits, workspace, p->workspace_bytes, (hipStream_t)stream);
}

int64_t moe_fp8_workspace_bytes(const moe_fp8_params* p) {
  if (!fp8_ok(p) || !split_ok(p->splits, 0) || !fp8_fast(p) || p->tile > kFp8GemmTiles) return 0;
  return workspace_of(kFp8GemmTileTable, kFp8GemmTiles, fp8_args(p), 128, p->tile, p->splits);
}

}  // extern "C"
