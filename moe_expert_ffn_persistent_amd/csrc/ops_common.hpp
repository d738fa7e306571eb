// Device helpers shared by the operators around the expert FFN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ffn_common.hpp"
#include "moe_ffn.h"

namespace moe {

// One expert's rows: rows r0 .. r0+Me-1, and which of its M-blocks this is.
struct Group {
  int e, m, r0, Me;
  bool ok;
};

// row_offset[i] of L experts, inside 0..rows whatever the array holds
__device__ __forceinline__ int clamped_offset(const int32_t* off, int L, int rows, int i) {
  return min(max(off[min(i, L)], 0), rows);
}

// The experts' M-blocks of TM rows, counted by every wavefront for itself: a
// lane looks at four experts (L <= 256), one prefix sum over the lanes.
template <int TM>
struct GroupScan {
  static_assert(MOE_MAX_LOCAL_EXPERTS <= 256, "four experts a lane");
  int o[5], t[4], excl, sum;
  int total;   // M-blocks of all experts

  __device__ __forceinline__ GroupScan(const int32_t* off, int L, int rows) {
    const int lane = threadIdx.x & 63;
    if (off == nullptr) L = 0;
#pragma unroll
    for (int j = 0; j < 5; ++j) o[j] = L == 0 ? 0 : clamped_offset(off, L, rows, lane * 4 + j);
    sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t[j] = (max(o[j + 1] - o[j], 0) + TM - 1) / TM;
      sum += t[j];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    excl = incl - sum;
    total = __builtin_amdgcn_readlane(incl, 63);
  }

  // M-block p (uniform); not ok past the last one
  __device__ __forceinline__ Group find(int p) const {
    const int lane = threadIdx.x & 63;
    int q = p - excl;
    const uint64_t hit = __ballot(q >= 0 && q < sum);
    Group g{0, 0, 0, 0, hit != 0};
    if (!g.ok) return g;
    int e = lane * 4, r0 = o[0], Me = o[1] - o[0];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const bool past = e == lane * 4 + j && q >= t[j];
      q -= past ? t[j] : 0;
      e += past;
      r0 = past ? o[j + 1] : r0;
      Me = past ? o[j + 2] - o[j + 1] : Me;
    }
    const int src = __builtin_ctzll(hit);
    g.e = __builtin_amdgcn_readlane(e, src);
    g.m = __builtin_amdgcn_readlane(q, src);
    g.r0 = __builtin_amdgcn_readlane(r0, src);
    g.Me = __builtin_amdgcn_readlane(Me, src);
    return g;
  }
};

// Tile of workgroup b, of `n`: workgroups go round-robin over the 8 XCDs, so
// runs of consecutive tiles are dealt to the XCDs in turn: tiles that run
// together on one XCD, and share operand rows in its L2, are neighbours. A run
// is 32 tiles (an XCD's compute units), fewer when that would leave XCDs
// without any: 64 tiles on two XCDs ran up to 2.1 times as long as on all. With
// no tiles (no expert has rows) the run is one, and every b lies past the end.
__device__ __forceinline__ int xcd_tile(int b, int n) {
  const int run = max(1, min(32, (n + 7) >> 3));
  const int x = b & 7, i = b >> 3, q = i / run;
  return (q * 8 + x) * run + i - q * run;
}

// Neighbouring tiles t of a grid of `mi` x `ni`: groups of four rows, column
// by column.
__device__ __forceinline__ void tile_at(int t, int mi, int ni, int& i, int& j) {
  const int g = t / (4 * ni), rem = t - g * 4 * ni;
  const int h = min(4, mi - g * 4);
  j = rem / h;
  i = g * 4 + rem - j * h;
}

// Range s of `splits` of a sum over nc, in whole stages of BK: where it starts
// and how much it adds up (nothing, if earlier ranges took all)
template <int BK>
__device__ __forceinline__ int split_range(int nc, int splits, int s, int& c0) {
  c0 = 0;
  if (splits == 1) return nc;
  const int stages = (nc + BK - 1) / BK, each = (stages + splits - 1) / splits * BK;
  c0 = min(s * each, nc);
  return min(nc - c0, each);
}

// Rows to work on: all of them, or row_offset[0] .. row_offset[L]-1.
__device__ __forceinline__ void row_range(const int32_t* off, int L, long long rows, int& lo, int& hi) {
  lo = off ? clamped_offset(off, L, (int)rows, 0) : 0;
  hi = off ? clamped_offset(off, L, (int)rows, L) : (int)rows;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return uint4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
}

// Eight consecutive elements of which the first n exist (the others read as
// zero, are not written). `vec`: the row is 16-byte aligned and n is 8.
__device__ __forceinline__ void load8(const __bf16* p, int n, bool vec, float (&x)[8]) {
  if (vec) {
    unpack8(*reinterpret_cast<const uint4*>(p), x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? (float)p[i] : 0.f;
  }
}

__device__ __forceinline__ void load8(const float* p, int n, bool vec, float (&x)[8]) {
  if (vec) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? p[i] : 0.f;
  }
}

__device__ __forceinline__ void store8(__bf16* p, int n, bool vec, const float (&x)[8]) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = pack8(x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (__bf16)x[i];
  }
}

// Block scale of values whose largest magnitude has the fp32 bits `amax`
// (taken as an integer maximum, which carries infinities and NaN along):
// fp32(amax / 448), 1 for a block of zeros or one whose quotient underflows.
__device__ __forceinline__ float block_scale(uint32_t amax) {
  const float s = __builtin_bit_cast(float, amax) / 448.f;
  return s == 0.f ? 1.f : s;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

// The e4m3 codes of fp32(x[i] / scale), ties to even, where the quotient is
// correctly rounded: with inv = 1/scale correctly rounded, q = x inv is off by
// less than 1.5 units in the last place, one correction q + inv (x - q scale)
// with fused multiply-adds brings it within one, and a second one then rounds
// correctly (Markstein's theorem). Without them codes differ: bf16 values
// over an amax of 8 bits land exactly on the border between two codes once in
// a few hundred. Scales so small that the residual's last bit (2^-47 of x)
// would fall below the smallest fp32 number, or whose reciprocal does, divide.
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float scale) {
  const float inv = 1.f / scale;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = x[i] * inv;
    y[i] = __builtin_fmaf(__builtin_fmaf(-y[i], scale, x[i]), inv, y[i]);
    y[i] = __builtin_fmaf(__builtin_fmaf(-y[i], scale, x[i]), inv, y[i]);
  }
  if (!(scale > 1e-26f && scale < 1e37f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] / scale;
  }
  const bool finite = abs_bits(scale) < 0x7f800000u;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(y[i], -448.f, 448.f);
  uint2 q{pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7])};
  if (!finite) q = uint2{0x7f7f7f7fu, 0x7f7f7f7fu};
  return q;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int n, bool vec, uint2 q) {
  if (vec) {
    *reinterpret_cast<uint2*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

// Integer maximum over 8 or 16 neighbouring lanes, all active (quantisation: a
// lane holds 16 or 8 of a block's 128 columns): quad permutations and mirrors of
// the lane row, no LDS.
__device__ __forceinline__ uint32_t max8(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));    // lane ^ 1
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));    // lane ^ 2
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));  // 7 - lane
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max8(v);
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true));  // 15 - lane
}

}  // namespace moe
