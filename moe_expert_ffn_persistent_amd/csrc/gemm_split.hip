// The joining of a product whose sum was cut into ranges (calls with few output
// tiles and a long sum, where whole tiles would leave compute units idle):
//
//   out(i, j) = sum over s of part_s(i, j), in ascending s, fp32
//
// One pass over the fp32 ranges, which the caches mostly still hold; the result
// does not depend on which workgroup finished first.
#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

// Eight columns a thread. Rows are the experts' (forward, dgrad), or the L * n
// rows of the weights (wgrad).
template <bool BF16>
__global__ void __launch_bounds__(256) moe_join_splits_k(const GemmArgs a, const float* ws) {
  const bool wgrad = a.op == MOE_GROUPED_WGRAD, fwd = a.op == MOE_GROUPED_FORWARD;
  int lo = 0, hi = a.L * a.n;
  if (!wgrad) row_range(a.row_offset, a.L, a.rows, lo, hi);
  const int nj = fwd ? a.n : a.k, pieces = nj / 8;
  const long long ld = wgrad ? a.ld_w : fwd ? a.ld_y : a.ld_x;
  void* const out = wgrad ? a.w : fwd ? a.y : a.x;
  const long long end = (long long)hi * pieces, step = (long long)gridDim.x * 256;
  for (long long p = (long long)lo * pieces + blockIdx.x * 256 + threadIdx.x; p < end; p += step) {
    const int r = (int)(p / pieces), c = (int)(p - (long long)r * pieces) * 8;
    long long at = (long long)r * ld + c;
    if (wgrad) {
      const int e = r / a.n;
      at = (long long)e * a.es_w + (long long)(r - e * a.n) * ld + c;
      // an expert without rows keeps what accumulates, to the bit
      if (a.accumulate && clamped_offset(a.row_offset, a.L, a.rows, e + 1) <= clamped_offset(a.row_offset, a.L, a.rows, e)) continue;
    }
    const float* src = ws + (long long)r * nj + c;
    float sum[8] = {};
    for (int s = 0; s < a.splits; ++s, src += a.part) {
      float x[8];
      load8(src, 8, true, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += x[i];
    }
    if constexpr (BF16) {
      __bf16* o = static_cast<__bf16*>(out) + at;
      if (a.accumulate) {
        float x[8];
        load8(o, 8, true, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += x[i];
      }
      store8(o, 8, true, sum);
    } else {
      float* o = static_cast<float*>(out) + at;
      if (a.accumulate) {
        float x[8];
        load8(o, 8, true, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += x[i];
      }
      reinterpret_cast<float4*>(o)[0] = float4{sum[0], sum[1], sum[2], sum[3]};
      reinterpret_cast<float4*>(o)[1] = float4{sum[4], sum[5], sum[6], sum[7]};
    }
  }
}

}  // namespace

GemmArgs split_args(const GemmArgs& a, float* ws) {
  GemmArgs b = a;
  b.out_bf16 = b.accumulate = false;
  switch (a.op) {
    case MOE_GROUPED_FORWARD:
      b.y = ws;
      b.ld_y = a.n;
      b.part = (long long)a.rows * a.n;
      break;
    case MOE_GROUPED_DGRAD:
      b.x = ws;
      b.ld_x = a.k;
      b.part = (long long)a.rows * a.k;
      break;
    default:
      b.w = ws;
      b.ld_w = a.k;
      b.es_w = (long long)a.n * a.k;
      b.part = a.L * b.es_w;
  }
  return b;
}

hipError_t launch_join_splits(const GemmArgs& a, const float* ws, hipStream_t s) {
  GemmArgs b = a;
  b.part = split_args(a, nullptr).part;
  const long long blocks = (b.part / 8 + 255) / 256;
  const unsigned grid = (unsigned)std::min<long long>(std::max<long long>(blocks, 1), 4096);
  if (a.out_bf16) moe_join_splits_k<true><<<grid, 256, 0, s>>>(b, ws);
  else moe_join_splits_k<false><<<grid, 256, 0, s>>>(b, ws);
  return hipGetLastError();
}

}  // namespace moe
