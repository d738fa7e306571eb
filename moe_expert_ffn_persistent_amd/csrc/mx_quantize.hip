// Quantisation to the OCP Microscaling (MX) formats: blocks of 32 consecutive
// elements of a row share one E8M0 scale byte s, a value is code * 2^(s - 127).
//
//   e = floor(log2(amax of the block)) - emax   (emax 8: e4m3, 2: e2m1; at least
//       -127; 0 for a block of zeros)
//   code = the format's value nearest to x / 2^e, ties to even, at most its largest
//
// One pass over the bytes, bound by HBM when large and by the launch when small.
#include <type_traits>

#include "internal.hpp"
#include "mx_common.hpp"

namespace moe {
namespace {

// A lane holds E columns of a block (32 / E lanes each). bf16 takes E = 16, two
// 16-byte loads; fp32 takes E = 8, since its loads would else lie 64 bytes apart.
template <class T, int E, bool E2M1, bool WHOLE>
__global__ void __launch_bounds__(256) moe_quantize_mx_k(const MxQuantArgs a, int tpr) {
  int lo, hi;
  row_range(a.row_offset, a.L, a.rows, lo, hi);
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr, rpw = 256 / tpr;
  const int kb = (a.cols + 31) / 32;
  const T* x0 = static_cast<const T*>(a.x) + (size_t)blockIdx.z * a.bs_x;
  uint8_t* q0 = a.codes + (size_t)blockIdx.z * a.bs_codes;
  uint8_t* s0 = a.scales + (size_t)blockIdx.z * a.bs_scales;
  for (long long r = lo + (long long)blockIdx.x * rpw + sub; r < hi; r += (long long)gridDim.x * rpw) {
    for (int c = (blockIdx.y * tpr + t) * E; c < kb * 32; c += gridDim.y * tpr * E) {   // alike for the lanes of a block
      float x[E];
      uint32_t mx = 0;
      load_cols<E, WHOLE>(x0 + r * a.ld_x, c, a.cols, x);
#pragma unroll
      for (int i = 0; i < E; ++i) mx = max(mx, abs_bits(x[i]));
      mx = E == 16 ? max2(mx) : max4(mx);
      const MxScale s = mx_scale<E2M1>(mx);
      store_mx<E2M1, E>(q0 + r * a.ld_codes, c, a.cols, x, s);
      if (t % (32 / E) == 0) s0[r * a.ld_scales + c / 32] = s.byte;
    }
  }
}

}  // namespace

hipError_t launch_quantize_mx(const MxQuantArgs& a, bool e2m1, bool fp32, hipStream_t s) {
  const int E = fp32 ? 8 : 16, pieces = (a.cols + E - 1) / E;
  int tpr = 32 / E;
  while (tpr < 256 && tpr < pieces) tpr *= 2;
  const long long need = (a.rows + 256 / tpr - 1) / (256 / tpr);
  const int y = (int)std::min<long long>((pieces + tpr - 1) / tpr, std::max<long long>(1, 1024 / need));
  const dim3 grid((unsigned)std::min<long long>(need, 4096), y, a.batch);
  auto run = [&](auto whole) {
    constexpr bool W = decltype(whole)::value;
    if (fp32) {
      if (e2m1) moe_quantize_mx_k<float, 8, true, W><<<grid, 256, 0, s>>>(a, tpr);
      else moe_quantize_mx_k<float, 8, false, W><<<grid, 256, 0, s>>>(a, tpr);
    } else {
      if (e2m1) moe_quantize_mx_k<__bf16, 16, true, W><<<grid, 256, 0, s>>>(a, tpr);
      else moe_quantize_mx_k<__bf16, 16, false, W><<<grid, 256, 0, s>>>(a, tpr);
    }
  };
  if (a.cols % 8 == 0) run(std::true_type{});
  else run(std::false_type{});
  return hipGetLastError();
}

}  // namespace moe
