// Rows of the local experts gathered from the tokens (dispatch) and each
// token's rows summed (combine): each other's gradients, both one pass over
// the bytes; and the gradients of the sum with a weight for each row.
#include <type_traits>

#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

// out[r] = x[row_pair[r] / k]. LPR lanes copy whole rows in pieces of V bytes a
// lane, several in flight. The grid is fixed and strides over the rows
// that exist: the layout's capacity (every pair local) is several times the
// rows routed here, and a workgroup for each would mostly start and end.
template <class V, int LPR>
__global__ void __launch_bounds__(256) moe_dispatch_rows_k(const RowsArgs a) {
  int lo, hi;
  row_range(a.row_offset, a.L, a.rows, lo, hi);
  auto first = [](int v) { return LPR == 64 ? uni(v) : v; };   // alike for the lanes of a row
  const int group = first((int)(blockIdx.x * (256 / LPR) + threadIdx.x / LPR));
  const int lane = threadIdx.x % LPR;
  const int n = a.hidden * a.elem / (int)sizeof(V);
  for (int r = lo + group; r < hi; r += gridDim.x * (256 / LPR)) {
    const int f = first(a.index[r]);
    const bool ok = f >= 0 && f < a.pairs;
    const V* src = reinterpret_cast<const V*>(static_cast<const char*>(a.in) + (size_t)(ok ? f / a.k : 0) * a.ld_in);
    V* dst = reinterpret_cast<V*>(static_cast<char*>(a.out) + (size_t)r * a.ld_out);
    int c = lane;
    for (; c + 3 * LPR < n; c += 4 * LPR) {
      V v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = ok ? src[c + LPR * j] : V{};
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[c + LPR * j] = v[j];
    }
    for (; c < n; c += LPR) dst[c] = ok ? src[c] : V{};
  }
}

// y[n] = sum of the token's rows, ascending slots, fp32; WEIGHTED: each times its
// pair's weight, one fused multiply-add. TPT threads take a
// token. A wavefront finds the slots that are local with one load and a ballot,
// so slots of other GPUs cost nothing, and a lane has eight columns of up to U
// pieces of the row in flight, of the next slot before this one's are added: 160
// us with one piece and one slot at a time, 90 us so (16384 tokens x 7168, 8
// slots of which one in the mean is local: 470 MB).
template <bool BF16, int TPT, int U, bool WEIGHTED, bool WHOLE>
__global__ void __launch_bounds__(256) moe_combine_rows_k(const RowsArgs a, const float* weights, int tokens) {
  const int n = blockIdx.x * (256 / TPT) + uni((int)threadIdx.x / TPT), lane = threadIdx.x & 63;
  if (n >= tokens) return;
  const int idx = lane < a.k ? a.index[(size_t)n * a.k + lane] : -1;
  const uint64_t local = __ballot(idx >= 0 && idx < a.rows);
  float weight = 1.f;
  if constexpr (WEIGHTED) weight = lane < a.k ? weights[(size_t)n * a.k + lane] : 0.f;
  char* yrow = static_cast<char*>(a.out) + (size_t)n * a.ld_out;
  for (int c0 = threadIdx.x % TPT * 8; c0 < a.hidden; c0 += U * TPT * 8) {
    auto load = [&](int slot, Raw<__bf16, WHOLE> (&v)[U]) {
      const int r = __builtin_amdgcn_readlane(idx, slot);
      const __bf16* row = reinterpret_cast<const __bf16*>(static_cast<const char*>(a.in) + (size_t)r * a.ld_in);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * TPT * 8;
        if (u && uni(c) >= a.hidden) break;   // no lane of this wavefront has any
        v[u].load(row, c, a.hidden);
      }
    };
    float s[U][8] = {};
    uint64_t left = local;
    Raw<__bf16, WHOLE> v[2][U];
    if (left) load(__builtin_ctzll(left), v[0]);
    while (left) {
      float w = 1.f;
      if constexpr (WEIGHTED) w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), __builtin_ctzll(left)));
      left &= left - 1;
      if (left) load(__builtin_ctzll(left), v[1]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u && uni(c0 + u * TPT * 8) >= a.hidden) break;
        float x[8];
        v[0][u].get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[u][i] = WEIGHTED ? __builtin_fmaf(w, x[i], s[u][i]) : s[u][i] + x[i];
        v[0][u] = v[1][u];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * TPT * 8, m = min(8, a.hidden - c);
      if (u && uni(c) >= a.hidden) break;
      if (m <= 0) continue;
      if constexpr (BF16) put8(reinterpret_cast<__bf16*>(yrow) + c, m, s[u]);
      else put8(reinterpret_cast<float*>(yrow) + c, m, s[u]);
    }
  }
}

// Gradients of the weighted sum y[n] = sum over j of w[n, j] rows[p(n, j)]:
//   drows[p(n, j)] = w[n, j] dy[n],  dw[n, j] = dy[n] . rows[p(n, j)]
// (0 where the slot is not local). TPT threads take a token: its dy is read
// once and held while its local rows pass (rows longer than U pieces of the
// threads read the rest of it again, from the caches), and a slot's dot product
// is joined over the lanes and, through LDS, over the wavefronts, in an order
// that sizes settle.
template <class D, int TPT, int U, bool WHOLE>
__global__ void __launch_bounds__(256) moe_combine_backward_k(const CombineBackwardArgs a) {
  __shared__ float part[4][16];
  const int sub = uni((int)threadIdx.x / TPT), n = blockIdx.x * (256 / TPT) + sub, lane = threadIdx.x & 63;
  const bool live = n < a.tokens;
  const int idx = live && lane < a.k ? a.pair_row[(size_t)n * a.k + lane] : -1;
  const float weight = live && lane < a.k ? a.weights[(size_t)n * a.k + lane] : 0.f;
  const uint64_t local = __ballot(idx >= 0 && idx < a.cap);
  float mine = 0.f;   // lane j: slot j's dot product, of this wavefront's columns
  if (local) {
    const D* dy = static_cast<const D*>(a.dy) + (size_t)n * a.ld_dy;
    const int t0 = threadIdx.x % TPT * 8;
    Raw<D, WHOLE> d[U];
    Raw<__bf16, WHOLE> x[2][U];
    auto load = [&](auto& to, const auto* row, int c0) {
#pragma unroll
      for (int u = 0; u < U; ++u) to[u].load(row, c0 + u * TPT * 8, a.hidden);
    };
    auto row_of = [&](int slot) { return static_cast<const __bf16*>(a.rows) + (size_t)__builtin_amdgcn_readlane(idx, slot) * a.ld_rows; };
    load(x[0], row_of(__builtin_ctzll(local)), t0);
    load(d, dy, t0);
    for (uint64_t left = local; left; left &= left - 1) {
      const int slot = __builtin_ctzll(left);
      const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), slot));
      const uint64_t more = left & (left - 1);
      if (more) load(x[1], row_of(__builtin_ctzll(more)), t0);   // the next row is on its way
      __bf16* drow = static_cast<__bf16*>(a.drows) + (size_t)__builtin_amdgcn_readlane(idx, slot) * a.ld_drows;
      float dot = 0.f;
      for (int c0 = t0; c0 < a.hidden; c0 += U * TPT * 8) {
        if (a.hidden > U * TPT * 8) {
          load(d, dy, c0);
          if (c0 != t0) load(x[0], row_of(slot), c0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * TPT * 8, m = min(8, a.hidden - c);
          float g[8], z[8];
          d[u].get(g);
          x[0][u].get(z);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot = __builtin_fmaf(g[i], z[i], dot);
            g[i] *= w;
          }
          if (m > 0) put8(drow + c, m, g);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) x[0][u] = x[1][u];
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) dot += __shfl_xor(dot, s, 64);
      if (lane == slot) mine = dot;
    }
  }
  if constexpr (TPT > 64) {
    if (lane < 16) part[threadIdx.x >> 6][lane] = mine;
    __syncthreads();
    mine = 0.f;
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < TPT / 64; ++i) mine += part[sub * (TPT / 64) + i][lane];
    }
  }
  if (live && threadIdx.x % TPT < a.k) a.dweights[(size_t)n * a.k + lane] = mine;
}

}  // namespace

hipError_t launch_dispatch_rows(const RowsArgs& a, hipStream_t s) {
  const uintptr_t bits = (uintptr_t)a.in | (uintptr_t)a.out | (uintptr_t)a.ld_in | (uintptr_t)a.ld_out |
                         (uintptr_t)((size_t)a.hidden * a.elem);
  auto run = [&](auto piece, auto lanes) {
    using V = decltype(piece);
    constexpr int LPR = decltype(lanes)::value;
    const long long rows = 256 / LPR;   // of a workgroup at a time
    moe_dispatch_rows_k<V, LPR><<<(unsigned)std::min<long long>((a.rows + rows - 1) / rows, 2048), 256, 0, s>>>(a);
  };
  // Short rows: a quarter of a wavefront each (100000 rows of 208 bytes 16.9 to
  // 9.3 us, of 640 bytes 22.0 to 21.3; 800 bytes 27.7 to 31.4).
  constexpr std::integral_constant<int, 64> wave{};
  if (bits % 16 == 0 && a.hidden * a.elem <= 640) run(uint4{}, std::integral_constant<int, 16>{});
  else if (bits % 16 == 0) run(uint4{}, wave);
  else if (bits % 4 == 0) run(uint32_t{}, wave);
  else if (bits % 2 == 0) run(uint16_t{}, wave);
  else run(uint8_t{}, wave);
  return hipGetLastError();
}

hipError_t launch_combine_rows(const RowsArgs& a, const float* weights, bool bf16_out, hipStream_t s) {
  const int tokens = (int)(a.pairs / a.k);
  auto run = [&](auto tpt, auto pieces) {
    constexpr int T = decltype(tpt)::value, U = decltype(pieces)::value;
    const int grid = (tokens + 256 / T - 1) / (256 / T);
    auto go = [&](auto bf16, auto whole) {
      constexpr bool B = decltype(bf16)::value, W = decltype(whole)::value;
      if (weights) moe_combine_rows_k<B, T, U, true, W><<<grid, 256, 0, s>>>(a, weights, tokens);
      else moe_combine_rows_k<B, T, U, false, W><<<grid, 256, 0, s>>>(a, nullptr, tokens);
    };
    auto type = [&](auto whole) {
      if (bf16_out) go(std::true_type{}, whole);
      else go(std::false_type{}, whole);
    };
    if (a.hidden % 8 == 0) type(std::true_type{});
    else type(std::false_type{});
    return hipGetLastError();
  };
  using std::integral_constant;
  // Few tokens take a workgroup each, whatever their length (8 slots, 4 tokens x
  // 4096: 4.7 us, with two wavefronts a token 5.9, with one 10); with many, short
  // rows take fewer threads, whose lanes all have columns (30000 tokens, one slot
  // of 8 local: 512 columns 11.4 us, a workgroup each 28.4; 1016: 20.6 and 37.8;
  // 2056: 39.9 and 56.2; 4096: 96.5 and 98.6; 7168: 167.5 and 165.3).
  if (tokens > 1024) {
    if (a.hidden <= 512) return run(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (a.hidden <= 1024) return run(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (a.hidden <= 4096) return run(integral_constant<int, 128>{}, integral_constant<int, 4>{});
  }
  return run(integral_constant<int, 256>{}, integral_constant<int, 4>{});
}

hipError_t launch_combine_backward(const CombineBackwardArgs& a, hipStream_t s) {
  auto run = [&](auto tpt, auto pieces) {
    constexpr int T = decltype(tpt)::value, U = decltype(pieces)::value;
    const int grid = (a.tokens + 256 / T - 1) / (256 / T);
    auto go = [&](auto whole) {
      constexpr bool W = decltype(whole)::value;
      if (a.dy_fp32) moe_combine_backward_k<float, T, U, W><<<grid, 256, 0, s>>>(a);
      else moe_combine_backward_k<__bf16, T, U, W><<<grid, 256, 0, s>>>(a);
    };
    if (a.hidden % 8 == 0) go(std::true_type{});
    else go(std::false_type{});
    return hipGetLastError();
  };
  using std::integral_constant;
  if (a.tokens > 1024) {
    if (a.hidden <= 512) return run(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (a.hidden <= 1024) return run(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (a.hidden <= 4096) return run(integral_constant<int, 128>{}, integral_constant<int, 4>{});
  }
  return run(integral_constant<int, 256>{}, integral_constant<int, 4>{});
}

}  // namespace moe
