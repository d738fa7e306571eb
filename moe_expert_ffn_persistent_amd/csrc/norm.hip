// RMS norm of the residual stream, forward with the stream's addition and the
// output in the format that the next product takes, and its gradients:
//
//   s = x + residual, rounded to the stream's type and stored
//   r = 1 / sqrt(mean over the row of s^2 + eps),  y = s r w
//
//   g = dy w,  dx = dresidual + r (g - s r^2 mean(g s)),  dw = sum over rows of dy s r
//
// One pass over the bytes: a row stays in the registers of its threads between
// its sums and what they scale. fp32 throughout. Bound by HBM when large and by
// the launch when small.
#include "internal.hpp"
#include "mx_common.hpp"

namespace moe {
namespace {

enum Kind { kPlain, kFp8, kMx };   // outputs without scales, e4m3 with fp32 scales, MX

__device__ __forceinline__ float rms_inv(float squares, int hidden, float eps) {
  return 1.f / sqrtf(squares / (float)hidden + eps);
}

// Sums of N values over the tpr threads of a row, to all of them. Rows of more
// than a wavefront join through `part`; every thread of the workgroup calls.
template <int N, int THREADS>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float (*part)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    for (int d = 1; d < min(tpr, 64); d <<= 1) v[k] += __shfl_xor(v[k], d, 64);
  if (tpr > 64) {
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) part[threadIdx.x >> 6][k] = v[k];
    __syncthreads();
    const int w0 = (threadIdx.x / tpr) * (tpr >> 6);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = 0.f;
    for (int i = 0; i < tpr / 64; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += part[w0 + i][k];
  }
}

// Eight columns of the weight (1 without one, 0 behind the row's end)
__device__ __forceinline__ void load_weight(const NormArgs& a, int c, float (&w)[8]) {
  const int m = min(8, a.hidden - c);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = i < m ? 1.f : 0.f;
  if (a.weight == nullptr || m <= 0) return;
  if (a.weight_fp32) get8(static_cast<const float*>(a.weight), c, a.hidden, w);
  else get8(static_cast<const __bf16*>(a.weight), c, a.hidden, w);
}

// Eight columns of the output. The lanes of a scale block (16, or 4) call together.
template <int KIND>
__device__ __forceinline__ void store_out(const NormArgs& a, long long r, int c, const float (&y)[8]) {
  const int m = min(8, a.hidden - c);
  if constexpr (KIND == kPlain) {
    if (m <= 0) return;
    if (a.format == MOE_NORM_BF16) put8(static_cast<__bf16*>(a.out) + r * a.ld_out + c, m, y);
    else put8(static_cast<float*>(a.out) + r * a.ld_out + c, m, y);
  } else {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, i < m ? abs_bits(y[i]) : 0u);
    uint8_t* row = static_cast<uint8_t*>(a.out) + r * a.ld_out;
    if constexpr (KIND == kFp8) {
      const float scale = block_scale(max16(mx));
      const uint2 q = quant8(y, scale);
      if (m == 8) *reinterpret_cast<u32x2u*>(row + c) = u32x2u{q.x, q.y};
      else if (m > 0) store_codes(row + c, m, false, q);
      if (c % 128 == 0 && m > 0) static_cast<float*>(a.scales)[r * a.ld_scales + c / 128] = scale;
    } else {
      mx = max4(mx);
      uint8_t byte;
      if (a.format == MOE_NORM_MX_E2M1) {
        const MxScale s = mx_scale<true>(mx);
        store_mx<true, 8>(row, c, a.hidden, y, s);
        byte = s.byte;
      } else {
        const MxScale s = mx_scale<false>(mx);
        store_mx<false, 8>(row, c, a.hidden, y, s);
        byte = s.byte;
      }
      if (c % 32 == 0 && m > 0) static_cast<uint8_t*>(a.scales)[r * a.ld_scales + c / 32] = byte;
    }
  }
}

// Rows of up to 8 P tpr columns: tpr threads take one, eight neighbouring
// columns a thread in each of P pieces.
template <class T, int KIND, int P, int THREADS, bool WHOLE>
__global__ void __launch_bounds__(THREADS) moe_rms_norm_k(const NormArgs a, int tpr) {
  __shared__ float part[2][THREADS / 64][1];
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr, rpw = THREADS / tpr;
  const long long step = (long long)gridDim.x * rpw;
  struct Row {
    Raw<T, WHOLE> x[P], res[P];
  } row, next;
  auto load = [&](Row& to, long long r) {
    const int cols = r < a.rows ? a.hidden : 0;
    const T *x = static_cast<const T*>(a.x) + r * a.ld_x, *res = static_cast<const T*>(a.residual) + r * a.ld_residual;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      to.x[p].load(x, (p * tpr + t) * 8, cols);
      if (a.residual) to.res[p].load(res, (p * tpr + t) * 8, cols);
    }
  };
  load(row, (long long)blockIdx.x * rpw + sub);
  float w[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p) load_weight(a, (p * tpr + t) * 8, w[p]);
  int odd = 0;
  for (long long base = (long long)blockIdx.x * rpw; base < a.rows; base += step, odd ^= 1) {
    const long long r = base + sub;
    const bool live = r < a.rows;
    if (base + step < a.rows) load(next, r + step);
    float v[P][8], sum[1] = {0.f};
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * tpr + t) * 8, m = live ? min(8, a.hidden - c) : 0;
      row.x[p].get(v[p]);
      if (a.residual) {
        float o[8];
        row.res[p].get(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] = (float)(T)(v[p][i] + o[i]);
        if (m > 0) {
          put8(static_cast<T*>(a.stream) + r * a.ld_stream + c, m, v[p]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(v[p][i], v[p][i], sum[0]);
    }
    row_sum<1, THREADS>(sum, tpr, part[odd]);
    const float inv = rms_inv(sum[0], a.hidden, a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * tpr + t) * 8;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v[p][i] * inv * w[p][i];
      // a row that is not there: its lanes take part in no other row's blocks
      if (live) store_out<KIND>(a, r, c, y);
    }
    row = next;
  }
}

// Rows of any length: two passes over them, the second reads the stored stream.
template <class T, int KIND>
__global__ void __launch_bounds__(1024) moe_rms_norm_long_k(const NormArgs a) {
  __shared__ float part[2][16][1];
  const T* in = static_cast<const T*>(a.stream ? a.stream : a.x);
  const long long ld = a.stream ? a.ld_stream : a.ld_x;
  int odd = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x, odd ^= 1) {
    float sum[1] = {0.f};
    for (int c = threadIdx.x * 8; c < a.hidden; c += 8192) {
      const int m = min(8, a.hidden - c);
      float v[8];
      get8(static_cast<const T*>(a.x) + r * a.ld_x, c, a.hidden, v);
      if (a.residual) {
        float o[8];
        get8(static_cast<const T*>(a.residual) + r * a.ld_residual, c, a.hidden, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)(T)(v[i] + o[i]);
        put8(static_cast<T*>(a.stream) + r * a.ld_stream + c, m, v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(v[i], v[i], sum[0]);
    }
    row_sum<1, 1024>(sum, 1024, part[odd]);
    const float inv = rms_inv(sum[0], a.hidden, a.eps);
    for (int c0 = 0; c0 < a.hidden; c0 += 8192) {   // every lane: scale blocks join theirs
      const int c = c0 + threadIdx.x * 8, m = min(8, a.hidden - c);
      float v[8], w[8];
      get8(in + r * ld, c, a.hidden, v);
      load_weight(a, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * w[i];
      store_out<KIND>(a, r, c, v);
    }
  }
}

// The gradients. A workgroup walks its rows, the next one on its way while one is
// summed, and keeps its part of dw in registers; the parts are joined by a second
// kernel, in their order.
template <class T, class D, int P, int THREADS, bool WHOLE>
__global__ void __launch_bounds__(THREADS, THREADS / 64 / 4) moe_rms_norm_backward_k(const NormArgs a, int tpr) {
  __shared__ float part[2][THREADS / 64][2];
  __shared__ float joined[P == 1 && THREADS == 256 ? THREADS * 8 : 1];
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr, rpw = THREADS / tpr;
  const long long step = (long long)gridDim.x * rpw;
  struct Row {
    Raw<T, WHOLE> x[P], add[P];
    Raw<D, WHOLE> dy[P];
  } row, next;
  constexpr bool AHEAD = P == 1;   // two pieces and their successors are too many registers
  auto load = [&](Row& to, long long r) {
    const int cols = r < a.rows ? a.hidden : 0;
    const T *x = static_cast<const T*>(a.x) + r * a.ld_x, *add = static_cast<const T*>(a.dresidual) + r * a.ld_dresidual;
    const D* dy = static_cast<const D*>(a.dy) + r * a.ld_dy;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      to.x[p].load(x, (p * tpr + t) * 8, cols);
      to.dy[p].load(dy, (p * tpr + t) * 8, cols);
      if (a.dresidual) to.add[p].load(add, (p * tpr + t) * 8, cols);
      else to.add[p] = {};
    }
  };
  if constexpr (AHEAD) load(row, (long long)blockIdx.x * rpw + sub);
  float w[P][8], dw[P][8] = {};
#pragma unroll
  for (int p = 0; p < P; ++p) load_weight(a, (p * tpr + t) * 8, w[p]);
  int odd = 0;
  for (long long base = (long long)blockIdx.x * rpw; base < a.rows; base += step, odd ^= 1) {
    const long long r = base + sub;
    const bool live = r < a.rows;
    if constexpr (!AHEAD) load(row, r);
    else if (base + step < a.rows) load(next, r + step);
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float v[8], d[8];
      row.x[p].get(v);
      row.dy[p].get(d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] = __builtin_fmaf(v[i], v[i], sum[0]);
        sum[1] = __builtin_fmaf(d[i] * w[p][i], v[i], sum[1]);
      }
    }
    row_sum<2, THREADS>(sum, tpr, part[odd]);
    const float inv = rms_inv(sum[0], a.hidden, a.eps);
    const float along = inv * inv * (sum[1] / (float)a.hidden);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * tpr + t) * 8, m = live ? min(8, a.hidden - c) : 0;
      float v[8], d[8], g[8];
      row.x[p].get(v);
      row.dy[p].get(d);
      row.add[p].get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = __builtin_fmaf(inv, d[i] * w[p][i] - v[i] * along, g[i]);
        dw[p][i] = __builtin_fmaf(d[i], live ? v[i] * inv : 0.f, dw[p][i]);
      }
      if (m > 0) {
        put8(static_cast<T*>(a.dx) + r * a.ld_dx + c, m, g);
      }
    }
    if constexpr (AHEAD) row = next;
  }
  if (!a.part) return;
  float* out = a.part + (long long)blockIdx.x * a.hidden;
  if (rpw > 1) {   // the rows of the workgroup that ran side by side (P is 1)
    if constexpr (P == 1 && THREADS == 256) {
#pragma unroll
      for (int i = 0; i < 8; ++i) joined[threadIdx.x * 8 + i] = dw[0][i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.hidden; c += THREADS) {
        float sum = 0.f;
        for (int s = 0; s < rpw; ++s) sum += joined[s * tpr * 8 + c];
        out[c] = sum;
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * tpr + t) * 8;
      if (c < a.hidden) put8(out + c, a.hidden - c, dw[p]);
    }
  }
}

template <class T, class D>
__global__ void __launch_bounds__(1024) moe_rms_norm_backward_long_k(const NormArgs a) {
  __shared__ float part[2][16][2];
  float* out = a.part ? a.part + (long long)blockIdx.x * a.hidden : nullptr;
  int odd = 0;
  bool first = true;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x, odd ^= 1) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
    const D* dy = static_cast<const D*>(a.dy) + r * a.ld_dy;
    float sum[2] = {0.f, 0.f};
    for (int c = threadIdx.x * 8; c < a.hidden; c += 8192) {
      const int m = min(8, a.hidden - c);
      float v[8], d[8], w[8];
      get8(x, c, a.hidden, v);
      get8(dy, c, a.hidden, d);
      load_weight(a, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] = __builtin_fmaf(v[i], v[i], sum[0]);
        sum[1] = __builtin_fmaf(d[i] * w[i], v[i], sum[1]);
      }
    }
    row_sum<2, 1024>(sum, 1024, part[odd]);
    const float inv = rms_inv(sum[0], a.hidden, a.eps);
    const float along = inv * inv * (sum[1] / (float)a.hidden);
    for (int c = threadIdx.x * 8; c < a.hidden; c += 8192) {
      const int m = min(8, a.hidden - c);
      float v[8], d[8], w[8], g[8], add[8] = {};
      get8(x, c, a.hidden, v);
      get8(dy, c, a.hidden, d);
      load_weight(a, c, w);
      if (a.dresidual) get8(static_cast<const T*>(a.dresidual) + r * a.ld_dresidual, c, a.hidden, add);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = __builtin_fmaf(inv, d[i] * w[i] - v[i] * along, add[i]);
        // this thread's own columns of the part
        if (out && i < m) out[c + i] = __builtin_fmaf(d[i], v[i] * inv, first ? 0.f : out[c + i]);
      }
      put8(static_cast<T*>(a.dx) + r * a.ld_dx + c, m, g);
    }
    first = false;
  }
}

// dw(c) = sum over the groups of part(g, c), ascending within 64 slices, then the
// slices: 16 columns a workgroup, four of them a thread, four groups of a slice in
// flight (with 16 slices of one at a time 512 groups of 4096 columns took 20 us).
__global__ void __launch_bounds__(256) moe_join_dweight_k(const float* part, float* dweight, int groups, int hidden) {
  __shared__ float slice[64][17];
  const int c0 = blockIdx.x * 16 + (threadIdx.x & 3) * 4, s = threadIdx.x >> 2;
  float sum[4] = {};
  for (int g = s; g < groups; g += 256) {
    float v[4][4] = {};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (g + 64 * u >= groups || c0 >= hidden) continue;
      const float* src = part + (long long)(g + 64 * u) * hidden + c0;
      if (c0 + 4 <= hidden) {
        const u32x4u x = *reinterpret_cast<const u32x4u*>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = __uint_as_float(x[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + i < hidden) v[u][i] = src[i];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += v[u][i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) slice[s][(threadIdx.x & 3) * 4 + i] = sum[i];
  __syncthreads();
  const int c = blockIdx.x * 16 + threadIdx.x;
  if (threadIdx.x < 16 && c < hidden) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) all += slice[i][threadIdx.x];
    dweight[c] = all;
  }
}

constexpr int kHeld = 16384;   // columns that 1024 threads hold in two pieces (four spill)

// Threads of a row that they hold in one piece: the least power of two, at least
// the lanes of a scale block. Rows of several pieces take the whole workgroup.
int threads_for(int hidden, int most) {
  int t = 16;
  while (t < most && t * 8 < hidden) t *= 2;
  return t;
}

// Threads of a workgroup, and the pieces of a row that each holds: few rows take a
// thread for each piece (128 x 7168: 4.9 us, with 256 threads of four pieces 6.7),
// many fewer, so that a compute unit holds several rows (16384 x 7168 forward 179 us,
// 190 with 1024 threads of one piece, 194 with 256 of four; to MX e4m3 163, 187, 255).
template <class F>
hipError_t with_shape(long long rows, int hidden, F f) {
  using std::integral_constant;
  constexpr integral_constant<int, 1> one{};
  constexpr integral_constant<int, 2> two{};
  if (hidden <= 2048) return f(one, integral_constant<int, 256>{});
  if (hidden <= 4096) return f(one, integral_constant<int, 512>{});
  if (hidden <= 8192) {
    if (rows <= 512) return f(one, integral_constant<int, 1024>{});
    return f(two, integral_constant<int, 512>{});
  }
  return f(two, integral_constant<int, 1024>{});
}

template <class T, int KIND>
hipError_t forward(const NormArgs& a, hipStream_t s) {
  if (a.hidden > kHeld) {
    moe_rms_norm_long_k<T, KIND><<<(unsigned)std::min<long long>(a.rows, 4 * kCus), 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  return with_shape(a.rows, a.hidden, [&](auto pieces, auto threads) {
    constexpr int P = decltype(pieces)::value, THREADS = decltype(threads)::value;
    const int tpr = P == 1 && THREADS == 256 ? threads_for(a.hidden, THREADS) : THREADS;
    const long long need = (a.rows + THREADS / tpr - 1) / (THREADS / tpr);
    const unsigned grid = (unsigned)std::min<long long>(need, kCus * 2048ll / THREADS);
    if (a.hidden % 8 == 0) moe_rms_norm_k<T, KIND, P, THREADS, true><<<grid, THREADS, 0, s>>>(a, tpr);
    else moe_rms_norm_k<T, KIND, P, THREADS, false><<<grid, THREADS, 0, s>>>(a, tpr);
    return hipGetLastError();
  });
}

template <class T>
hipError_t forward_kind(const NormArgs& a, hipStream_t s) {
  switch (a.format) {
    case MOE_NORM_BF16:
    case MOE_NORM_FP32: return forward<T, kPlain>(a, s);
    case MOE_NORM_FP8: return forward<T, kFp8>(a, s);
  }
  return forward<T, kMx>(a, s);
}

template <class T, class D>
hipError_t backward(const NormArgs& a, hipStream_t s) {
  const int groups = norm_backward_groups(a.rows, a.hidden, a.fp32);
  if (a.hidden > kHeld) {
    moe_rms_norm_backward_long_k<T, D><<<groups, 1024, 0, s>>>(a);
  } else {
    with_shape(a.rows, a.hidden, [&](auto pieces, auto threads) {
      constexpr int P = decltype(pieces)::value, THREADS = decltype(threads)::value;
      const int tpr = P == 1 && THREADS == 256 ? threads_for(a.hidden, THREADS) : THREADS;
      if (a.hidden % 8 == 0) moe_rms_norm_backward_k<T, D, P, THREADS, true><<<groups, THREADS, 0, s>>>(a, tpr);
      else moe_rms_norm_backward_k<T, D, P, THREADS, false><<<groups, THREADS, 0, s>>>(a, tpr);
      return hipSuccess;
    });
  }
  if (a.part && a.part != a.dweight) moe_join_dweight_k<<<(a.hidden + 15) / 16, 256, 0, s>>>(a.part, a.dweight, groups, a.hidden);
  return hipGetLastError();
}

}  // namespace

// As many as the compute units hold at once by their registers (16384 x 7168 bf16: 186
// us with two a unit, 217 with one; fp32 8192 x 7168: 171 and 164). Beyond one a unit
// only with some rows each, since a part is as long as a row in fp32 (1024 x 7168: 23
// us with 256, 30 with 512).
int norm_backward_groups(long long rows, int hidden, bool fp32) {
  const int rpw = hidden <= 2048 ? 256 / threads_for(hidden, 256) : 1;
  const int each = hidden <= 2048 ? 4 : hidden <= 4096 ? 2 : hidden <= 8192 && !fp32 ? 2 : 1;
  const long long need = (rows + rpw - 1) / rpw;
  // one launch instead of two where a workgroup takes its rows in as little time (2 x
  // 4096: 5.7 us, 8.4 in two launches; 4 x 4096: 8.9 and 8.4; 16 x 512: 7.8 and 8.5)
  if (need <= 2 || (hidden <= 512 && need <= 4)) return 1;
  return (int)std::min<long long>(each * kCus, std::max(std::min<long long>(need, kCus), need / (hidden <= 2048 ? 2 : 4)));
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  return a.fp32 ? forward_kind<float>(a, s) : forward_kind<__bf16>(a, s);
}

hipError_t launch_rms_norm_backward(const NormArgs& a, hipStream_t s) {
  if (a.fp32) return a.format == MOE_NORM_FP32 ? backward<float, float>(a, s) : backward<float, __bf16>(a, s);
  return a.format == MOE_NORM_FP32 ? backward<__bf16, float>(a, s) : backward<__bf16, __bf16>(a, s);
}

}  // namespace moe
