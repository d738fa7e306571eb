// Grouped matrix products for any sizes, strides and alignment: the kernel of
// the calls the 16-byte kernels cannot take (odd row lengths, unaligned
// pointers), and the plainest statement of the three products:
//
//   out(i, j) = sum over c of A(i, c) B(j, c)
//   forward  i = row, j = n, c = k      A = x, B = W[e]
//   dgrad    i = row, j = k, c = n      A = y, B = W[e]^T
//   wgrad    i = n,   j = k, c = row    A = y^T, B = x^T
//
// 64 x 64 tiles, four wavefronts of one 32 x 32 block each. Elements are read
// one by one with bounds checks along the operand's unit-stride axis, staged
// in LDS as bf16 and multiplied by v_mfma_f32_32x32x16_bf16; e4m3 values are
// exact in bf16, their block sums are taken per 128 columns and scaled by the
// VALU. Bound by the element loads; the sizes that matter take other kernels.
#include <type_traits>

#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

constexpr int kAnyTile = 64, kAnyBK = 32, kAnyLd = kAnyBK + 8;

__device__ __forceinline__ __bf16 element(const __bf16* p) { return *p; }
__device__ __forceinline__ __bf16 element(const uint8_t* p) {
  return (__bf16)__builtin_amdgcn_cvt_f32_fp8((int)*p, 0);
}

// 64 x 32 elements of the operand at (i0, c0) to LDS; outside ni x nc: zero.
template <class T>
__device__ __forceinline__ void stage_any(const T* p, long long si, long long sc, int i0, int c0, int ni, int nc,
                                          __bf16* lds) {
  const int tid = threadIdx.x;
  const bool rowwise = sc == 1;
  const int i1 = rowwise ? tid >> 2 : (tid & 7) * 8;
  const int c1 = rowwise ? (tid & 3) * 8 : tid >> 3;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = rowwise ? i1 : i1 + j, c = rowwise ? c1 + j : c1;
    const bool in = i0 + i < ni && c0 + c < nc;
    lds[i * kAnyLd + c] = in ? element(p + (i0 + i) * si + (c0 + c) * sc) : (__bf16)0.f;
  }
}

template <bool FP8>
__global__ void __launch_bounds__(256) moe_gemm_any(const GemmArgs a) {
  using T = typename std::conditional<FP8, uint8_t, __bf16>::type;
  __shared__ __attribute__((aligned(16))) __bf16 as[kAnyTile * kAnyLd];
  __shared__ __attribute__((aligned(16))) __bf16 bs[kAnyTile * kAnyLd];
  const bool wgrad = a.op == MOE_GROUPED_WGRAD, fwd = a.op == MOE_GROUPED_FORWARD;
  Group g;
  int i0;
  if (wgrad) {
    const int nt = (a.n + kAnyTile - 1) / kAnyTile;
    g.e = blockIdx.x / nt;
    i0 = (blockIdx.x - g.e * nt) * kAnyTile;
    g.r0 = clamped_offset(a.row_offset, a.L, a.rows, g.e);
    g.Me = max(clamped_offset(a.row_offset, a.L, a.rows, g.e + 1) - g.r0, 0);
    if (a.accumulate && g.Me == 0) return;   // an expert without rows keeps what accumulates, to the bit
  } else if (a.row_offset) {
    g = GroupScan<kAnyTile>(a.row_offset, a.L, a.rows).find(blockIdx.x);
    if (!g.ok) return;
    i0 = g.m * kAnyTile;
  } else {
    g = Group{0, 0, 0, a.rows, true};
    i0 = blockIdx.x * kAnyTile;
  }
  const int j0 = blockIdx.y * kAnyTile;
  const T* x = static_cast<const T*>(a.x) + (size_t)g.r0 * a.ld_x;
  const T* y = static_cast<const T*>(a.y) + (size_t)g.r0 * a.ld_y;
  const T* w = static_cast<const T*>(a.w) + (size_t)g.e * a.es_w;
  const T* A = fwd ? x : y;
  const T* B = wgrad ? x : w;
  const int ni = wgrad ? a.n : g.Me, nj = fwd ? a.n : a.k, nc = fwd ? a.k : wgrad ? g.Me : a.n;
  const long long sai = wgrad ? 1 : fwd ? a.ld_x : a.ld_y, sac = wgrad ? a.ld_y : 1;
  const long long sbj = fwd ? a.ld_w : 1, sbc = fwd ? 1 : wgrad ? a.ld_x : a.ld_w;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wi = (wave & 1) * 32, wj = (wave >> 1) * 32;
  const int j = j0 + wj + (lane & 31);
  f32x16 acc = f32x16{}, part = f32x16{};
  const int kb = (nc + 127) / 128;
  for (int c0 = 0; c0 < nc; c0 += kAnyBK) {
    __syncthreads();
    stage_any(A, sai, sac, i0, c0, ni, nc, as);
    stage_any(B, sbj, sbc, j0, c0, nj, nc, bs);
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < kAnyBK / 16; ++ks) {
      const int at = (lane & 31) * kAnyLd + ks * 16 + (lane >> 5) * 8;
      const bf16x8 fa = *reinterpret_cast<const bf16x8*>(as + wi * kAnyLd + at);
      const bf16x8 fb = *reinterpret_cast<const bf16x8*>(bs + wj * kAnyLd + at);
      part = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, part, 0, 0, 0);
    }
    if constexpr (FP8) {
      // the end of a 128-wide block: its scales
      if ((c0 & 127) == 128 - kAnyBK || c0 + kAnyBK >= nc) {
        const int b = c0 >> 7;
        const float sw = j < nj ? a.ws[((size_t)g.e * ((a.n + 127) / 128) + j / 128) * kb + b] : 0.f;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int i = i0 + wi + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
          const float sx = i < ni ? a.xs[(size_t)(g.r0 + i) * a.ld_xs + b] : 0.f;
          acc[v] += part[v] * (sx * sw);
        }
        part = f32x16{};
      }
    }
  }
  if constexpr (!FP8) acc = part;
  if (j >= nj) return;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int i = i0 + wi + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
    if (i >= ni) continue;
    const size_t at = wgrad ? (size_t)g.e * a.es_w + (size_t)i * a.ld_w + j
                            : (size_t)(g.r0 + i) * (fwd ? a.ld_y : a.ld_x) + j;
    void* out = wgrad ? a.w : fwd ? a.y : a.x;
    if (a.out_bf16) {
      __bf16* o = static_cast<__bf16*>(out) + at;
      *o = (__bf16)(a.accumulate ? acc[v] + (float)*o : acc[v]);
    } else {
      float* o = static_cast<float*>(out) + at;
      *o = a.accumulate ? acc[v] + *o : acc[v];
    }
  }
}

}  // namespace

hipError_t launch_gemm_any(const GemmArgs& a, bool fp8, hipStream_t s) {
  const bool wgrad = a.op == MOE_GROUPED_WGRAD;
  const int nj = a.op == MOE_GROUPED_FORWARD ? a.n : a.k;
  const long long blocks = wgrad ? (long long)a.L * ((a.n + kAnyTile - 1) / kAnyTile)
                                 : ((long long)a.rows + (long long)a.L * (kAnyTile - 1)) / kAnyTile;
  const dim3 grid((unsigned)blocks, (nj + kAnyTile - 1) / kAnyTile);
  if (fp8) moe_gemm_any<true><<<grid, 256, 0, s>>>(a);
  else moe_gemm_any<false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
