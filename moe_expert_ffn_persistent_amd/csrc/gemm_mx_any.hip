// Matrix product of MX operands of any alignment (rows of any byte, odd sums):
//
//   y(r, n) = sum over blocks b of 32 along k of 2^(xs(r, b) + ws(n, b) - 254)
//             sum over k in b of x(r, k) w(n, k)
//
// A wavefront computes 16 rows x 16 features with v_mfma_scale_f32_16x16x128,
// which applies both blocks' scales itself; its fragments come straight from memory,
// where rows end byte by byte. For what the tile kernels cannot load (8192 x 7168 x
// 4096, e4m3 rows on odd bytes: 10.0 ms, e2m1 7.0).
//
// Operand placement of the instruction (checked on the GPU with scaled one-hot
// operands): lane l holds row l % 16. A lane of e2m1 values holds the 32 elements
// of block q = l / 16, in nibble order, under its own scale byte. A lane of e4m3
// values holds elements 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q + 15, and its
// scale byte is that of block q. Result: lane l, value v: row l % 16 of B,
// feature 4 (l / 16) + v of A.
#include <climits>

#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

// 16 bytes of a row from byte `at`, of which those before `end` exist; `odd`: the
// last of them holds one e2m1 code in its low bits
__device__ __forceinline__ uint4 bytes16(const uint8_t* row, int at, int end, bool odd) {
  if (at + 16 <= end && !odd) {
    const u32x4u v = *reinterpret_cast<const u32x4u*>(row + at);
    return uint4{v.x, v.y, v.z, v.w};
  }
  uint32_t w[4] = {};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (at + i >= end) continue;
    uint32_t b = row[at + i];
    if (odd && at + i == end - 1) b &= 0x0f;
    w[i / 4] |= b << (8 * (i & 3));
  }
  return uint4{w[0], w[1], w[2], w[3]};
}

template <bool X4>
__global__ void __launch_bounds__(256) moe_gemm_mx_any(const GemmArgs a) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const bool grouped = a.row_offset != nullptr;
  const GroupScan<16> scan(a.row_offset, grouped ? a.L : 0, a.rows);
  const int ti = grouped ? scan.total : (a.rows + 15) / 16, tj = (a.n + 15) / 16;
  const long long tiles = (long long)ti * tj;
  const int kb = (a.k + 31) / 32, wbytes = (a.k + 1) / 2, xbytes = X4 ? wbytes : a.k;
  const bool odd = a.k & 1;
  for (long long tile = (long long)blockIdx.x * 4 + uni((int)(threadIdx.x >> 6)); tile < tiles; tile += (long long)gridDim.x * 4) {
    const int i = (int)(tile / tj), j = (int)(tile - (long long)i * tj);
    const Group g = grouped ? scan.find(i) : Group{0, i, 0, a.rows, true};
    const int row = g.m * 16 + r16, feature = j * 16 + r16;
    const long long xr = g.r0 + min(row, g.Me - 1), wn = min(feature, a.n - 1);
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + xr * a.ld_x;
    const uint8_t* xs = reinterpret_cast<const uint8_t*>(a.xs) + xr * a.ld_xs;
    const uint8_t* w = static_cast<const uint8_t*>(a.w) + g.e * a.es_w + wn * a.ld_w;
    const uint8_t* ws = reinterpret_cast<const uint8_t*>(a.ws) + g.e * a.es_ws + wn * a.ld_ws;
    f32x4 acc{};
    for (int k0 = 0; k0 < a.k; k0 += 128) {
      const int b = k0 / 32 + q;
      const int sx = b < kb ? xs[b] : 127, sw = b < kb ? ws[b] : 127;   // nothing counts behind the end, a NaN scale would
      const uint4 wv = bytes16(w, k0 / 2 + 16 * q, wbytes, odd);
      const i32x8 af{(int)wv.x, (int)wv.y, (int)wv.z, (int)wv.w, 0, 0, 0, 0};
      const uint4 lo = bytes16(x, X4 ? k0 / 2 + 16 * q : k0 + 16 * q, xbytes, X4 && odd);
      const uint4 hi = X4 ? uint4{0, 0, 0, 0} : bytes16(x, k0 + 64 + 16 * q, xbytes, false);
      const i32x8 bf{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af, bf, acc, 4, X4 ? 4 : 0, 0, sw, 0, sx);
    }
    if (row >= g.Me) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int n = j * 16 + 4 * q + v;
      if (n >= a.n) continue;
      const long long at = (long long)(g.r0 + row) * a.ld_y + n;
      if (a.out_bf16) static_cast<__bf16*>(a.y)[at] = (__bf16)acc[v];
      else static_cast<float*>(a.y)[at] = acc[v];
    }
  }
}

}  // namespace

hipError_t launch_gemm_mx_any(const GemmArgs& a, hipStream_t s) {
  const long long mi = a.row_offset ? ((long long)a.rows + (long long)a.L * 15) / 16 : (a.rows + 15) / 16;
  const long long tiles = mi * ((a.n + 15) / 16);
  const unsigned grid = (unsigned)std::min<long long>((tiles + 3) / 4, 1 << 20);
  if (a.x_e2m1) moe_gemm_mx_any<true><<<grid, 256, 0, s>>>(a);
  else moe_gemm_mx_any<false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
