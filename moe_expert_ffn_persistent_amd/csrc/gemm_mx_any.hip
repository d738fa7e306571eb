// Matrix product of MX operands of any alignment (rows of any byte, odd sums):
//
//   y(r, n) = sum over blocks b of 32 along k of 2^(xs(r, b) + ws(n, b) - 254)
//             sum over k in b of x(r, k) w(n, k)
//
// A wavefront computes 16 rows x 16 features, or 64 x 64, with
// v_mfma_scale_f32_16x16x128, which applies both blocks' scales itself; its fragments
// come straight from memory, whole 16 bytes of any alignment, and byte by byte at the
// ends of rows. For what the tile kernels cannot load (8192 x 7168 x 4096, e4m3 rows on
// odd bytes: 2.8 ms, e2m1 2.0).
//
// Operand placement of the instruction (checked on the GPU with scaled one-hot
// operands): lane l holds row l % 16. A lane of e2m1 values holds the 32 elements
// of block q = l / 16, in nibble order, under its own scale byte. A lane of e4m3
// values holds elements 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q + 15, and its
// scale byte is that of block q. Result: lane l, value v: row l % 16 of B,
// feature 4 (l / 16) + v of A.
#include <climits>
#include <type_traits>

#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

// 16 bytes of a row from byte `at`, of which those before `end` exist; `odd`: the
// last of them holds one e2m1 code in its low bits
__device__ __forceinline__ uint4 bytes16(const uint8_t* row, int at, int end, bool odd) {
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

__device__ __forceinline__ uint4 whole16(const uint8_t* p) {
  const u32x4u v = *reinterpret_cast<const u32x4u*>(p);
  return uint4{v.x, v.y, v.z, v.w};
}

// B x B blocks of 16 rows x 16 features a wavefront
template <bool X4, int B>
__global__ void __launch_bounds__(256) moe_gemm_mx_any(const GemmArgs a) {
  constexpr int T = 16 * B;
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const bool grouped = a.row_offset != nullptr;
  const GroupScan<T> scan(a.row_offset, grouped ? a.L : 0, a.rows);
  const int ti = grouped ? scan.total : (a.rows + T - 1) / T, tj = (a.n + T - 1) / T;
  const long long tiles = (long long)ti * tj;
  const int kb = (a.k + 31) / 32, wbytes = (a.k + 1) / 2, xbytes = X4 ? wbytes : a.k;
  const bool odd = a.k & 1;
  for (long long tile = (long long)blockIdx.x * 4 + uni((int)(threadIdx.x >> 6)); tile < tiles; tile += (long long)gridDim.x * 4) {
    const int i = (int)(tile / tj), j = (int)(tile - (long long)i * tj);
    const Group g = grouped ? scan.find(i) : Group{0, i, 0, a.rows, true};
    const uint8_t *x[B], *xs[B], *w[B], *ws[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const long long xr = g.r0 + min(g.m * T + b * 16 + r16, g.Me - 1), wn = min(j * T + b * 16 + r16, a.n - 1);
      x[b] = static_cast<const uint8_t*>(a.x) + xr * a.ld_x;
      xs[b] = reinterpret_cast<const uint8_t*>(a.xs) + xr * a.ld_xs;
      w[b] = static_cast<const uint8_t*>(a.w) + g.e * a.es_w + wn * a.ld_w;
      ws[b] = reinterpret_cast<const uint8_t*>(a.ws) + g.e * a.es_ws + wn * a.ld_ws;
    }
    f32x4 acc[B][B] = {};
    auto step = [&](int k0, auto full) {
      constexpr bool FULL = decltype(full)::value;
      const int kq = k0 / 32 + q, wat = k0 / 2 + 16 * q, xat = X4 ? wat : k0 + 16 * q;
      i32x8 af[B], bf[B];
      int sx[B], sw[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        sx[b] = FULL || kq < kb ? xs[b][kq] : 127;   // nothing counts behind the end, a NaN scale would
        sw[b] = FULL || kq < kb ? ws[b][kq] : 127;
        const uint4 wv = FULL ? whole16(w[b] + wat) : bytes16(w[b], wat, wbytes, odd);
        const uint4 lo = FULL ? whole16(x[b] + xat) : bytes16(x[b], xat, xbytes, X4 && odd);
        uint4 hi{0, 0, 0, 0};
        if constexpr (!X4) hi = FULL ? whole16(x[b] + xat + 64) : bytes16(x[b], xat + 64, xbytes, false);
        af[b] = i32x8{(int)wv.x, (int)wv.y, (int)wv.z, (int)wv.w, 0, 0, 0, 0};
        bf[b] = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
      }
#pragma unroll
      for (int f = 0; f < B; ++f)
#pragma unroll
        for (int r = 0; r < B; ++r)
          acc[f][r] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af[f], bf[r], acc[f][r], 4, X4 ? 4 : 0, 0, sw[f], 0, sx[r]);
    };
    int k0 = 0;
    for (; k0 + 128 <= a.k; k0 += 128) step(k0, std::true_type{});
    if (k0 < a.k) step(k0, std::false_type{});
#pragma unroll
    for (int r = 0; r < B; ++r) {
      const int row = g.m * T + r * 16 + r16;
      if (row >= g.Me) continue;
#pragma unroll
      for (int f = 0; f < B; ++f)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int n = j * T + f * 16 + 4 * q + v;
          if (n >= a.n) continue;
          const long long at = (long long)(g.r0 + row) * a.ld_y + n;
          if (a.out_bf16) static_cast<__bf16*>(a.y)[at] = (__bf16)acc[f][r][v];
          else static_cast<float*>(a.y)[at] = acc[f][r][v];
        }
    }
  }
}

template <int B>
hipError_t launch_any(const GemmArgs& a, hipStream_t s) {
  constexpr int T = 16 * B;
  const long long mi = a.row_offset ? ((long long)a.rows + (long long)a.L * (T - 1)) / T : (a.rows + T - 1) / T;
  const long long tiles = mi * ((a.n + T - 1) / T);
  const unsigned grid = (unsigned)std::min<long long>((tiles + 3) / 4, 1 << 20);
  if (a.x_e2m1) moe_gemm_mx_any<true, B><<<grid, 256, 0, s>>>(a);
  else moe_gemm_mx_any<false, B><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

// 4 x 4 blocks read a quarter as much, once they are wavefronts enough (7168 to 4096
// of e4m3 rows on odd bytes: 64 rows 345 us, 89 in single blocks; 256 rows, 256
// wavefronts, 346 and 342; 8192 rows 2.8 ms and 10.0)
hipError_t launch_gemm_mx_any(const GemmArgs& a, hipStream_t s) {
  const long long large = (a.expected + 63ll) / 64 * ((a.n + 63) / 64);
  return large > kCus && a.expected >= 32ll * a.L ? launch_any<4>(a, s) : launch_any<1>(a, s);
}

}  // namespace moe
