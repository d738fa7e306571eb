// SwiGLU of routed rows with the router weight, its gradients, and the
// quantisation of rows and weights to e4m3 with fp32 block scales: one pass
// over the bytes each, bound by HBM.
#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

// Threads of one row: the least power of two that covers its pieces of E
// columns, from `least` (the lanes of a scale block) to 256.
int threads_per_row(int cols, int E, int least) {
  int t = least;
  while (t < 256 && t * E < cols) t *= 2;
  return t;
}

// Workgroups along the rows and, where those are few, along the columns
// (`pieces` of them a row) of kernels that need no more than a scale block of a
// row at once: 16 x 7168 SwiGLU to e4m3 5.6 us without, 4.6 with.
dim3 row_grid(long long rows, int tpr, int pieces, int batch) {
  const long long need = (rows + 256 / tpr - 1) / (256 / tpr);
  const int y = (int)std::min<long long>((pieces + tpr - 1) / tpr, std::max<long long>(1, 1024 / need));
  return dim3((unsigned)std::min<long long>(need, 4096), y, batch);
}

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.f + __expf(-g)); }

// Eight columns a lane (16 in the e4m3 form, as in moe_quantize_rows_k, were 8 to
// 18% slower: twice the exponentials' registers).
template <bool FP8>
__global__ void __launch_bounds__(256) moe_swiglu_k(const SwigluArgs a, int tpr) {
  int lo, hi;
  row_range(a.row_offset, a.L, a.rows, lo, hi);
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr, rpw = 256 / tpr;
  const int I = a.inter, cols = (I + 127) & ~127;
  for (long long r = lo + (long long)blockIdx.x * rpw + sub; r < hi; r += (long long)gridDim.x * rpw) {
    const __bf16* g = static_cast<const __bf16*>(a.a) + r * a.ld_a;
    const float w = a.weight ? a.weight[r] : 1.f;
    for (int c = (blockIdx.y * tpr + t) * 8; c < cols; c += gridDim.y * tpr * 8) {
      const int m = min(8, I - c);
      const bool v = a.vec && m == 8;
      float gx[8] = {}, ux[8] = {}, h[8];
      if (m > 0) {
        load8(g + c, m, v, gx);
        load8(g + I + c, m, v, ux);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = gx[i] * sigmoid(gx[i]) * ux[i] * w;
      if constexpr (FP8) {
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = max(mx, i < m ? abs_bits(h[i]) : 0u);
        const float scale = block_scale(max16(mx));
        if (m > 0) store_codes(static_cast<uint8_t*>(a.h) + r * a.ld_h + c, m, v, quant8(h, scale));
        if ((t & 15) == 0) a.scales[r * a.ld_scales + c / 128] = scale;
      } else {
        if (m > 0) store8(static_cast<__bf16*>(a.h) + r * a.ld_h + c, m, v, h);
      }
    }
  }
}

__global__ void __launch_bounds__(256) moe_swiglu_backward_k(const SwigluArgs a, int tpr) {
  __shared__ float part[4];
  int lo, hi;
  row_range(a.row_offset, a.L, a.rows, lo, hi);
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr, rpw = 256 / tpr;
  const int I = a.inter;
  // every thread of the workgroup runs the same number of rounds: the row sum
  // of 128 and 256 threads goes through LDS behind barriers
  for (long long base = lo + (long long)blockIdx.x * rpw; base < hi; base += (long long)gridDim.x * rpw) {
    const long long r = base + sub;
    const bool live = r < hi;
    float dw = 0.f;
    if (live) {
      const __bf16* g = static_cast<const __bf16*>(a.a) + r * a.ld_a;
      const __bf16* dhp = static_cast<const __bf16*>(a.dh) + r * a.ld_h;
      __bf16* da = static_cast<__bf16*>(a.da) + r * a.ld_da;
      const float w = a.weight ? a.weight[r] : 1.f;
      for (int c = t * 8; c < I; c += tpr * 8) {
        const int m = min(8, I - c);
        const bool v = a.vec && m == 8;
        float gx[8], ux[8], d[8], dg[8], du[8];
        load8(g + c, m, v, gx);
        load8(g + I + c, m, v, ux);
        load8(dhp + c, m, v, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float s = sigmoid(gx[i]), act = gx[i] * s, back = d[i] * w;
          dw += d[i] * (act * ux[i]);
          du[i] = back * act;
          // s (1 + g (1 - s)) = s + act (1 - s)
          dg[i] = back * ux[i] * (s + act * (1.f - s));
        }
        store8(da + c, m, v, dg);
        store8(da + I + c, m, v, du);
      }
    }
    if (a.dweight) {
      for (int d = 1; d < min(tpr, 64); d <<= 1) dw += __shfl_xor(dw, d, 64);
      if (tpr > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dw;
        __syncthreads();
        const int w0 = (sub * tpr) >> 6;
        dw = 0.f;
        for (int i = 0; i < tpr / 64; ++i) dw += part[w0 + i];
      }
      if (live && t == 0) a.dweight[r] = dw;
    }
  }
}

// 1 x 128 blocks: a lane holds E columns of one (128/E lanes a block). bf16
// takes E = 16, a 16-byte store of codes each: with eight columns a lane the
// scale's two divisions and the maximum over the lanes were a third of the work
// (16384 x 7168: 87 us, 4.0 TB/s, against 72 us, 4.9 TB/s). fp32 takes E = 8,
// since 16 would spread a load over 64-byte strides (126 against 119 us).
template <class T, int E>
__global__ void __launch_bounds__(256) moe_quantize_rows_k(const QuantArgs a, int tpr) {
  int lo, hi;
  row_range(a.row_offset, a.L, a.rows, lo, hi);
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr, rpw = 256 / tpr;
  const int cb = (a.cols + 127) / 128;
  const T* x0 = static_cast<const T*>(a.x) + (size_t)blockIdx.z * a.bs_x;
  uint8_t* q0 = static_cast<uint8_t*>(a.codes) + (size_t)blockIdx.z * a.bs_codes;
  float* s0 = a.scales + (size_t)blockIdx.z * a.rows * cb;
  for (long long r = lo + (long long)blockIdx.x * rpw + sub; r < hi; r += (long long)gridDim.x * rpw) {
    for (int c = (blockIdx.y * tpr + t) * E; c < cb * 128; c += gridDim.y * tpr * E) {   // alike for the lanes of a block
      float x[E / 8][8] = {};
      uint32_t mx = 0;
#pragma unroll
      for (int h = 0; h < E / 8; ++h) {
        const int m = min(8, a.cols - c - 8 * h);
        if (m > 0) load8(x0 + r * a.ld_x + c + 8 * h, m, a.vec && m == 8, x[h]);
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = max(mx, abs_bits(x[h][i]));
      }
      const float scale = block_scale(E == 16 ? max8(mx) : max16(mx));
      uint8_t* q = q0 + r * a.ld_codes + c;
      uint2 codes[E / 8];
#pragma unroll
      for (int h = 0; h < E / 8; ++h) codes[h] = quant8(x[h], scale);
      if (E == 16 && a.vec16 && c + 16 <= a.cols) {
        *reinterpret_cast<uint4*>(q) = uint4{codes[0].x, codes[0].y, codes[E / 8 - 1].x, codes[E / 8 - 1].y};
      } else {
#pragma unroll
        for (int h = 0; h < E / 8; ++h) {
          const int m = min(8, a.cols - c - 8 * h);
          if (m > 0) store_codes(q + 8 * h, m, a.vec && m == 8, codes[h]);
        }
      }
      if (t % (128 / E) == 0) s0[r * cb + c / 128] = scale;
    }
  }
}

// 128 x 128 blocks: a workgroup holds one in registers, so it is read once; with
// 512 threads four pieces of eight columns each. The quotients are the longest
// part of a small call: 256 threads took 5.8 us where these take 4.4 (1000 x 104
// bf16), 70.5 against 66.8 at 16384 x 7168; 1024 gain no more on the small and
// lose up to 15% in between.
template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS) moe_quantize_blocks_k(const QuantArgs a) {
  constexpr int P = 16384 / 8 / THREADS, WAVES = THREADS / 64;   // pieces a thread
  __shared__ uint32_t part[WAVES];
  const int cb = (a.cols + 127) / 128, rb = (int)((a.rows + 127) / 128);
  const int bc = blockIdx.x % cb, br = blockIdx.x / cb;
  const T* x0 = static_cast<const T*>(a.x) + (size_t)blockIdx.y * a.bs_x;
  uint8_t* q0 = static_cast<uint8_t*>(a.codes) + (size_t)blockIdx.y * a.bs_codes;
  const int c = bc * 128 + (threadIdx.x & 15) * 8;
  const int m = min(8, a.cols - c);
  const bool v = a.vec && m == 8;
  const long long r0 = (long long)br * 128 + (threadIdx.x >> 4);
  float x[P][8] = {};
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const long long r = r0 + THREADS / 16 * j;
    if (r < a.rows && m > 0) load8(x0 + r * a.ld_x + c, m, v, x[j]);
  }
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, abs_bits(x[j][i]));
  mx = max16(mx);
  mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, 64));
  mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = mx;
  __syncthreads();
  mx = part[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) mx = max(mx, part[i]);
  const float scale = block_scale(mx);
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const long long r = r0 + THREADS / 16 * j;
    if (r < a.rows && m > 0) store_codes(q0 + r * a.ld_codes + c, m, v, quant8(x[j], scale));
  }
  if (threadIdx.x == 0) a.scales[((size_t)blockIdx.y * rb + br) * cb + bc] = scale;
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, bool fp8, hipStream_t s) {
  const int tpr = threads_per_row(a.inter, 8, fp8 ? 16 : 8);
  const dim3 grid = row_grid(a.rows, tpr, (a.inter + 7) / 8, 1);
  if (fp8) moe_swiglu_k<true><<<grid, 256, 0, s>>>(a, tpr);
  else moe_swiglu_k<false><<<grid, 256, 0, s>>>(a, tpr);
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(const SwigluArgs& a, hipStream_t s) {
  const int tpr = threads_per_row(a.inter, 8, 8);
  moe_swiglu_backward_k<<<row_grid(a.rows, tpr, 1, 1), 256, 0, s>>>(a, tpr);
  return hipGetLastError();
}

hipError_t launch_quantize(const QuantArgs& a, int block_rows, bool fp32, hipStream_t s) {
  if (block_rows == 1) {
    const int E = fp32 ? 8 : 16, tpr = threads_per_row(a.cols, E, 128 / E);
    const dim3 grid = row_grid(a.rows, tpr, (a.cols + E - 1) / E, a.batch);
    if (fp32) moe_quantize_rows_k<float, 8><<<grid, 256, 0, s>>>(a, tpr);
    else moe_quantize_rows_k<__bf16, 16><<<grid, 256, 0, s>>>(a, tpr);
  } else {
    const dim3 grid((unsigned)(((a.rows + 127) / 128) * ((a.cols + 127) / 128)), a.batch);
    constexpr int THREADS = 512;
    if (fp32) moe_quantize_blocks_k<float, THREADS><<<grid, THREADS, 0, s>>>(a);
    else moe_quantize_blocks_k<__bf16, THREADS><<<grid, THREADS, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
