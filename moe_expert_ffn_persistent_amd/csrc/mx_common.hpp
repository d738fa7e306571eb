// The OCP Microscaling formats on the device: block scales, codes, stores.
#pragma once

#include "ops_common.hpp"

namespace moe {

struct MxScale {
  uint8_t byte;   // E8M0
  float inv;      // 2^-(byte - 127), exact; 0 where the block has no scale
};

// Scale of a block whose largest magnitude has the fp32 bits `amax` (an integer
// maximum, which carries infinities and NaN along): floor(log2(amax)) is its
// exponent field, below the normal numbers the lowest scale is taken anyway. A
// block with an infinity or NaN has the NaN scale.
template <bool E2M1>
__device__ __forceinline__ MxScale mx_scale(uint32_t amax) {
  const int field = (int)(amax >> 23), e = max(field - (E2M1 ? 2 : 8), 0);   // e + 127
  if (field == 255) return MxScale{255, 0.f};
  if (amax == 0) return MxScale{127, 1.f};
  // 2^(127 - e): exponent field 254 - e, which e <= 254 - 2 keeps normal
  return MxScale{(uint8_t)e, __builtin_bit_cast(float, (uint32_t)(254 - e) << 23)};
}

// Codes of eight values: multiplied by the power of two (exact; what falls below
// the normal numbers is far below the formats' smallest step), kept to the
// format's largest value and rounded to the nearest even code.
__device__ __forceinline__ uint2 mx_e4m3x8(const float* x, const MxScale& s) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(x[i] * s.inv, -448.f, 448.f);
  const uint2 q{pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7])};
  return s.byte == 255 ? uint2{0x7f7f7f7fu, 0x7f7f7f7fu} : q;
}

// e2m1 has no NaN: the codes of a block without a scale are zeros
__device__ __forceinline__ uint32_t mx_e2m1x8(const float* x, const MxScale& s) {
  uint32_t q = 0;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(x[i] * s.inv, -6.f, 6.f);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[0], y[1], 1.f, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[2], y[3], 1.f, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[4], y[5], 1.f, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[6], y[7], 1.f, 3);
  return s.byte == 255 ? 0u : q;
}

// Columns c .. c+E-1 of a row of `cols` elements (zeros past its end)
template <int E, bool WHOLE, class T>
__device__ __forceinline__ void load_cols(const T* row, int c, int cols, float (&x)[E]) {
  Raw<T, WHOLE> r[E / 8];
#pragma unroll
  for (int h = 0; h < E / 8; ++h) r[h].load(row, c + 8 * h, cols);
#pragma unroll
  for (int h = 0; h < E / 8; ++h) {
    float v[8];
    r[h].get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[8 * h + i] = v[i];
  }
}

// Codes of columns c .. c+E-1 (c a multiple of E) of a row of `cols` elements,
// into the row's bytes. An odd row's last byte has zeros in its high bits.
template <bool E2M1, int E>
__device__ __forceinline__ void store_mx(uint8_t* row, int c, int cols, const float (&x)[E], const MxScale& s) {
  const int n = cols - c;
  if (n <= 0) return;
  if constexpr (E2M1) {
    uint32_t q[E / 8];
#pragma unroll
    for (int h = 0; h < E / 8; ++h) q[h] = mx_e2m1x8(x + 8 * h, s);
    uint8_t* p = row + c / 2;
    if (n >= E) {
      if constexpr (E == 16) *reinterpret_cast<u32x2u*>(p) = u32x2u{q[0], q[1]};
      else *reinterpret_cast<u32u*>(p) = q[0];
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i)
        if (2 * i < n) p[i] = (uint8_t)(q[i / 4] >> (8 * (i & 3))) & (2 * i + 1 < n ? 0xff : 0x0f);
    }
  } else {
    uint2 q[E / 8];
#pragma unroll
    for (int h = 0; h < E / 8; ++h) q[h] = mx_e4m3x8(x + 8 * h, s);
    uint8_t* p = row + c;
    if (n >= E) {
      if constexpr (E == 16) *reinterpret_cast<u32x4u*>(p) = u32x4u{q[0].x, q[0].y, q[1].x, q[1].y};
      else *reinterpret_cast<u32x2u*>(p) = u32x2u{q[0].x, q[0].y};
    } else {
#pragma unroll
      for (int h = 0; h < E / 8; ++h)
        if (n > 8 * h) store_codes(p + 8 * h, min(8, n - 8 * h), false, q[h]);
    }
  }
}

// Integer maximum over 2 or 4 neighbouring lanes, all active
__device__ __forceinline__ uint32_t max2(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));   // lane ^ 1
}
__device__ __forceinline__ uint32_t max4(uint32_t v) {
  v = max2(v);
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));   // lane ^ 2
}

}  // namespace moe
