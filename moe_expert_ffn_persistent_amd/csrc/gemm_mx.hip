// Matrix products of MX operands, dense or grouped by expert, for operands on
// whole 16 bytes (scales on four):
//
//   y(r, n) = sum over blocks b of 32 along k of 2^(xs(r, b) + ws(n, b) - 254)
//             sum over k in b of x(r, k) w(n, k)
//
// w is e2m1, x e4m3 or e2m1. v_mfma_scale_f32_16x16x128_f8f6f4 applies both
// blocks' E8M0 scales itself, so a sum stays in the matrix core's accumulators from
// the first k to the last. Weights are the A operand and rows the B operand: a
// lane's results are one row and runs of four consecutive n.
//
// A stage is 128 bytes of each row of x: 128 k of e4m3 beside 64-byte weight rows,
// or 256 k of e2m1 beside 128-byte ones (two MFMAs a 16 x 16 block), and the scale
// words of both (a word is 128 k). An NS-deep LDS ring is filled by direct-to-LDS
// copies between the MFMAs of an earlier stage. A ragged last stage is zeros in
// LDS, with scales of 1.
#include <climits>
#include <type_traits>

#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

// 16 bytes a lane from base + voff (bytes) to LDS m0 + 16 * lane; s_nop: m0's
// wait state (see dma16 in ffn_common.hpp)
__device__ __forceinline__ void dma16s(uint32_t voff, const char* base, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(m0) : "memory", "m0");
}

// KW > 1: KW wavefronts split the sum: a ring each, sums joined in LDS.
template <bool X4_, int TM_, int TN_, int WT_, int WF_, int NS_, int SP_, int OCC_, int KW_ = 1>
struct CfgM {
  static constexpr bool X4 = X4_;
  static constexpr int TM = TM_, TN = TN_, WT = WT_, WF = WF_, NS = NS_, SP = SP_, OCC = OCC_;
  static constexpr int KW = KW_, NW = WT * WF, THREADS = 64 * NW * KW;
  static constexpr int KS = X4 ? 256 : 128, H = KS / 128;          // k of a stage, MFMAs of a block in it
  static constexpr int FROW = KS / 2, TROW = 128;                  // bytes of a row in a stage
  static constexpr int TT = TM / WT, FT = TN / WF;
  static constexpr int TB = TT / 16, FB = FT / 16, NB = TB * FB;   // 16 x 16 blocks of a wavefront
  static constexpr int TP = TB > 1 ? TB / 2 : 1;                   // 32-row blocks
  static constexpr int NIT = TM * TROW / 1024 / NW, NIF = TN * FROW / 1024 / NW;
  static constexpr int WORDS = (TN + TM) * H;                      // scale words: weights' rows, then x's, for each 128 k
  static constexpr int NSC = (WORDS + 64 * NW - 1) / (64 * NW);
  static constexpr int NI = NIT + NIF + NSC;
  static constexpr int F_BYTES = TN * FROW, T_BYTES = TM * TROW, S_BYTES = NSC * NW * 256;
  static constexpr int STAGE = F_BYTES + T_BYTES + S_BYTES;
  static constexpr int EPI = NW * 16 * FT * 4;
  static constexpr int RING = NS * STAGE;
  static constexpr int LDS = KW * RING;
  static_assert(RING - STAGE >= EPI || KW > 1, "the epilogue stages behind the next tile's first stage");
  static_assert(KW == 1 || (NW == 1 && TM <= 32), "split wavefronts hold the whole tile each");
  static_assert(KW == 1 || RING >= TM * TN * 4, "a wavefront's sums fit its ring");
  // copies of a stage when only ntp 32-row blocks a wavefront hold rows, the scales' last
  static constexpr int copies(int ntp) { return NIF + NIT * ntp / TP + NSC; }
  static constexpr int issue_slot(int i, int nb, int ni) { return i * nb * SP / (ni * 8); }
  static_assert(NIT % TP == 0, "copies of a row block");
  static_assert(16 * FT * 2 % 1024 == 0 || KW > 1, "a 16-row piece of the epilogue is whole stores");
  static_assert(TB == 2 * TP - (TB == 1), "blocks of a wavefront");
  static_assert((TM * TROW) % (1024 * NW) == 0 && (TN * FROW) % (1024 * NW) == 0, "copies split evenly");
  static_assert(NS >= 2 && NI * (NS - 1) <= 63, "vmcnt range");
  static_assert(LDS * OCC <= 160 * 1024, "LDS");
};

// Physical 16-byte chunk of logical chunk c in row r of a stage, and back: a
// fragment read takes one chunk (4 h + lane / 16, or lane / 16) of 16 rows, and
// these bijections spread it over the banks.
template <int ROW>
__device__ __forceinline__ int chunk_at(int r, int c) {
  if constexpr (ROW == 64) return c ^ ((r >> 2) & 3) ^ ((c & 1) << 1);
  else return c ^ ((r >> 1) & 7);
}
template <int ROW>
__device__ __forceinline__ int chunk_in(int r, int p) {
  if constexpr (ROW == 64) {
    const int x = p ^ ((r >> 2) & 3);
    return x ^ ((x & 1) << 1);
  } else {
    return p ^ ((r >> 1) & 7);
  }
}

template <class C>
struct TileM {
  const char *fbase, *tbase;
  const char* sp[C::NSC];   // this lane's scale word of the first stage
  uint32_t fv[C::NIF], tv[C::NIT];
  f32x4 acc[C::FB][C::TB];

  __device__ __forceinline__ static int wave_of() { return C::NW == 1 ? 0 : uni((int)(threadIdx.x >> 6)); }

  // row and logical chunk of a lane in copy i of rows of ROW bytes
  template <int ROW>
  __device__ __forceinline__ static void place(int i, int& r, int& c) {
    constexpr int N = ROW / 16;
    const int lane = threadIdx.x & 63;
    r = (wave_of() + C::NW * i) * (1024 / ROW) + lane / N;
    c = chunk_in<ROW>(r, lane % N);
  }

  template <int ROW, int NI>
  __device__ __forceinline__ static void offsets(uint32_t (&v)[NI], long long ld, int last) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      int r, c;
      place<ROW>(i, r, c);
      v[i] = (uint32_t)min(r, last) * (uint32_t)ld + c * 16;
    }
  }

  // word q of a stage's scales: which 128 k of it, and which row
  __device__ __forceinline__ static int scale_word(int i) { return min((i * C::NW + wave_of()) * 64 + (int)(threadIdx.x & 63), C::WORDS - 1); }

  __device__ __forceinline__ void issue(int i, int kt, uint32_t slot) const {
    const uint32_t wave = wave_of();
    slot = uni(slot);
    if (i < C::NIF) {
      dma16s(fv[i], fbase + (long long)kt * C::FROW, slot + (wave + C::NW * i) * 1024);
    } else if (i < C::NIF + C::NIT) {
      dma16s(tv[i - C::NIF], tbase + (long long)kt * C::TROW, slot + C::F_BYTES + (wave + C::NW * (i - C::NIF)) * 1024);
    } else {
      const int s = i - C::NIF - C::NIT;
      dma4<kCacheNormal>(sp[s] + (long long)kt * (4 * C::H), slot + C::F_BYTES + C::T_BYTES + (s * C::NW + wave) * 256);
    }
  }

  // 16 bytes at `src` of which `n` e4m3 bytes (PACKED: e2m1 codes) exist
  template <bool PACKED>
  __device__ __forceinline__ static uint4 partial(const char* src, int n) {
    uint64_t v[2] = {0, 0};
    const int bytes = PACKED ? (n + 1) / 2 : n;
#pragma unroll 1
    for (int b = 0; b < bytes; ++b) {
      uint64_t x = (uint8_t)src[b];
      if (PACKED && 2 * b + 1 == n) x &= 0x0f;
      x <<= 8 * (b & 7);
      if (b < 8) v[0] |= x;
      else v[1] |= x;
    }
    return uint4{(uint32_t)v[0], (uint32_t)(v[0] >> 32), (uint32_t)v[1], (uint32_t)(v[1] >> 32)};
  }

  template <int ROW, bool PACKED>
  __device__ __forceinline__ void tail_copy(int i, int copy, const char* src, int kt, int left, char* dst) const {
    constexpr int E = PACKED ? 32 : 16;   // elements of 16 bytes
    int r, c;
    place<ROW>(i, r, c);
    const int have = left - c * E;
    char* at = dst + (wave_of() + C::NW * i) * 1024 + (threadIdx.x & 63) * 16;
    if (have >= E) issue(copy, kt, (uint32_t)(uintptr_t)(copy < C::NIF ? dst : dst - C::F_BYTES));
    else *reinterpret_cast<uint4*>(at) = have > 0 ? partial<PACKED>(src, have) : uint4{0, 0, 0, 0};
  }

  // the last stage when it holds only `left` < KS k
  __device__ __forceinline__ void issue_tail(int kt, int left, char* slot) const {
#pragma unroll
    for (int i = 0; i < C::NIF; ++i)
      tail_copy<C::FROW, true>(i, i, fbase + (long long)kt * C::FROW + fv[i], kt, left, slot);
#pragma unroll
    for (int i = 0; i < C::NIT; ++i)
      tail_copy<C::TROW, C::X4>(i, C::NIF + i, tbase + (long long)kt * C::TROW + tv[i], kt, left, slot + C::F_BYTES);
    // a scale of 1 for blocks that are not there: what lies behind the row may be NaN
    const int blocks = (left + 31) / 32;
#pragma unroll
    for (int i = 0; i < C::NSC; ++i) {
      const int h = scale_word(i) / (C::TN + C::TM);
      const uint8_t* src = reinterpret_cast<const uint8_t*>(sp[i]) + (long long)kt * (4 * C::H);
      uint32_t w = 0x7f7f7f7fu;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (4 * h + b < blocks) w = (w & ~(0xffu << (8 * b))) | (uint32_t)src[b] << (8 * b);
      *reinterpret_cast<uint32_t*>(slot + C::F_BYTES + C::T_BYTES + (i * C::NW + wave_of()) * 256 + (threadIdx.x & 63) * 4) = w;
    }
  }

  // A fragment of e2m1 rows, and of x's
  __device__ __forceinline__ static i32x8 frag_w(const char* stage, int r, int h, int q) {
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * C::FROW + (chunk_at<C::FROW>(r, 4 * h + q) << 4));
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
  }
  // e4m3: elements 16 q .. and 64 + 16 q .., which meet the weights' 32 q ..
  // (operand placement: gemm_mx_any.hip)
  __device__ __forceinline__ static i32x8 frag_x(const char* ts, int r, int h, int q) {
    const char* row = ts + r * C::TROW;
    const uint4 lo = *reinterpret_cast<const uint4*>(row + (chunk_at<C::TROW>(r, 4 * h + q) << 4));
    if constexpr (C::X4) return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, 0, 0, 0, 0};
    const uint4 hi = *reinterpret_cast<const uint4*>(row + (chunk_at<C::TROW>(r, 4 + q) << 4));
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  }

  // One stage. Only the first NTP of the wavefront's 32-row blocks are multiplied.
  template <bool COPY, int NTP>
  __device__ __forceinline__ void compute(const char* stage, int wf, int wt, int kt_next, uint32_t slot) {
    constexpr int TB = C::TB == 1 ? 1 : 2 * NTP, NB = C::FB * TB, NI = C::copies(NTP);
    // row of 16-row block j: 32-row blocks go to the row wavefronts in turn
    auto row = [&](int j) { return ((j >> 1) * C::WT + wt) * 32 + (j & 1) * 16; };
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    const char* ts = stage + C::F_BYTES;
    const uint8_t* sc = reinterpret_cast<const uint8_t*>(ts + C::T_BYTES) + r16 * 4 + q;
    i32x8 af[C::FB], bf[2];
    int sa[C::FB], sb[2];
    auto load_w = [&](int i, int h) {
      af[i] = frag_w(stage, wf * C::FT + i * 16 + r16, h, q);
      sa[i] = sc[(h * (C::TN + C::TM) + wf * C::FT + i * 16) * 4];
    };
    auto load_x = [&](int jj) {   // block jj of the stage's H * TB
      const int h = jj / TB, r = row(jj % TB);
      bf[jj & 1] = frag_x(ts, r + r16, h, q);
      sb[jj & 1] = sc[(h * (C::TN + C::TM) + C::TN + r) * 4];
    };
    load_x(0);
    load_w(0, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < C::H * NB; ++b) {
      const int jj = b / C::FB, j = jj % TB, h = jj / TB, i = b % C::FB;
      if (b + 1 < C::FB) load_w(b + 1, 0);
      if (i == 0 && jj + 1 < C::H * TB) load_x(jj + 1);
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af[i], bf[jj & 1], acc[i][j], 4, C::X4 ? 4 : 0, 0, sa[i], 0,
                                                                   sb[jj & 1]);
      if (j == TB - 1 && h + 1 < C::H) load_w(i, h + 1);
      if constexpr (COPY) {
#pragma unroll
        for (int k = 0; k < NI; ++k)
          if (C::issue_slot(k, C::H * NB, NI) == b) issue(k + C::NSC >= NI ? C::NI - NI + k : k, kt_next, slot);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Copies of the first stage (with KW > 1, the wavefront's first)
  __device__ __forceinline__ void first(char* lds, int K, int kw) const {
    if (kw < K / C::KS) {
#pragma unroll
      for (int i = 0; i < C::NI; ++i) issue(i, kw, (uint32_t)(uintptr_t)lds);
    } else if (kw == K / C::KS && K % C::KS) {
      issue_tail(kw, K % C::KS, lds);
    }
  }

  // All of K (with KW > 1, stages kw, kw + KW, ...), the first stage's copies
  // already issued
  template <int NTP>
  __device__ __forceinline__ void mainloop(char* lds, int K, int wf, int wt, int kw, int stores, bool fresh) {
    constexpr int NI = C::copies(NTP);
#pragma unroll
    for (int i = 0; i < C::FB; ++i)
#pragma unroll
      for (int j = 0; j < C::TB; ++j) acc[i][j] = f32x4{};
    const uint32_t ring = (uint32_t)(uintptr_t)lds;
    const int all = K / C::KS;
    const int left = all % C::KW == kw ? K % C::KS : 0;
    const int full = C::KW == 1 ? all : (all - kw + C::KW - 1) / C::KW;
    const int nk = full + (left != 0);
    auto at = [&](int s) { return C::KW == 1 ? s : kw + C::KW * s; };
    // without stores since the first stage's copies (fresh) all stages are on
    // their way at once, and counted below
    if (!fresh) wait_first(stores);
    if constexpr (C::NS > 2) {
      // past the previous tile's staging
      if constexpr (C::KW == 1) {
        if (!fresh) lds_barrier();
      }
#pragma unroll
      for (int s = 1; s < C::NS - 1; ++s) {
        if (s < full) {
#pragma unroll
          for (int i = 0; i < NI; ++i) issue(i + C::NSC >= NI ? C::NI - NI + i : i, at(s), ring + s * C::STAGE);
        } else if (s < nk) {
          issue_tail(at(s), left, lds + s * C::STAGE);
        }
      }
    }
    int slot = 0;
    const int nmain = full - (C::NS - 1);
    for (int s = 0; s < nmain; ++s) {
      if (s || fresh) vm_wait<NI * (C::NS - 2)>();   // the stage has landed (later ones may not have)
      if constexpr (C::KW == 1) lds_barrier();
      const int nslot = slot == 0 ? C::NS - 1 : slot - 1;
      compute<true, NTP>(lds + slot * C::STAGE, wf, wt, at(s + C::NS - 1), ring + nslot * C::STAGE);
      slot = slot + 1 == C::NS ? 0 : slot + 1;
    }
    for (int s = max(nmain, 0); s < nk; ++s) {
      if (s == 0 && !fresh) {
      } else if (left) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      else vm_wait_ahead<NI, C::NS - 2>(nk - 1 - s);
      if constexpr (C::KW == 1) lds_barrier();
      if (left && s + C::NS - 1 == full) issue_tail(at(full), left, lds + (full % C::NS) * C::STAGE);
      compute<false, NTP>(lds + slot * C::STAGE, wf, wt, 0, 0);
      slot = slot + 1 == C::NS ? 0 : slot + 1;
    }
  }

  // The tile's `rows` rows (at least one)
  __device__ __forceinline__ void multiply(char* lds, int rows, int K, int wf, int wt, int kw, int stores, bool fresh) {
    const int blocks = (min(rows, C::TM) + 32 * C::WT - 1) / (32 * C::WT);
    if constexpr (C::TB >= 4) {
      if (blocks == 1) return mainloop<1>(lds, K, wf, wt, kw, stores, fresh);
    }
    if constexpr (C::TB >= 6) {
      if (blocks == 2) return mainloop<2>(lds, K, wf, wt, kw, stores, fresh);
    }
    if constexpr (C::TB >= 8) {
      if (blocks == 3) return mainloop<3>(lds, K, wf, wt, kw, stores, fresh);
    }
    mainloop<C::TP>(lds, K, wf, wt, kw, stores, fresh);
  }

  // The first stage's copies have landed. They were issued before the previous
  // tile's `stores` stores (0: any number), and memory operations are counted
  // back in order: the stores may stay in flight.
  __device__ __forceinline__ static void wait_first(int stores) {
    static_assert(STORES<false> <= 63, "vmcnt range");
    if (stores == STORES<true>) vm_wait<STORES<true>>();
    else if (stores == STORES<false>) vm_wait<STORES<false>>();
    else vm_wait<0>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  // N columns of a row to `p`, of which those before `left` exist; vec: whole rows
  // are aligned for it
  template <int N, class T>
  __device__ __forceinline__ static void put(T* p, const T* v, int left, bool vec) {
    if (vec && left >= N) {
      using V = typename std::conditional<N * sizeof(T) == 16, uint4, uint2>::type;
      *reinterpret_cast<V*>(p) = *reinterpret_cast<const V*>(v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) p[i] = v[i];
    }
  }

  // KW > 1: the wavefronts' sums to LDS, joined in their order and written out.
  __device__ __forceinline__ void store_split(char* lds, void* out, long long ld, int i0, int ni, int j0, int nj, int kw,
                                              bool bf16, bool vec) {
    constexpr int ROWB = C::TN * 4, NCH = ROWB / 16;
    const int lane = threadIdx.x & 63;
    char* mine = lds + kw * C::RING;
#pragma unroll
    for (int i = 0; i < C::FB; ++i)
#pragma unroll
      for (int j = 0; j < C::TB; ++j)
        *reinterpret_cast<float4*>(mine + stage_off<ROWB>(j * 16 + (lane & 15), (i * 16 + 4 * (lane >> 4)) * 4)) =
            float4{acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
    __syncthreads();
    for (int idx = threadIdx.x; idx < C::TM * NCH; idx += C::THREADS) {
      const int r = idx / NCH, c = idx - r * NCH, i = i0 + r, col = j0 + c * 4;
      if (i >= ni || col >= nj) continue;
      float4 s = *reinterpret_cast<const float4*>(lds + stage_off<ROWB>(r, c * 16));
#pragma unroll
      for (int w = 1; w < C::KW; ++w) {
        const float4 o = *reinterpret_cast<const float4*>(lds + w * C::RING + stage_off<ROWB>(r, c * 16));
        s = float4{s.x + o.x, s.y + o.y, s.z + o.z, s.w + o.w};
      }
      const long long p = (long long)i * ld + col;
      if (bf16) {
        __attribute__((aligned(8))) const uint32_t v[2] = {pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w)};
        put<4>(static_cast<uint16_t*>(out) + p, reinterpret_cast<const uint16_t*>(v), nj - col, vec);
      } else {
        __attribute__((aligned(16))) const uint32_t v[4] = {__float_as_uint(s.x), __float_as_uint(s.y), __float_as_uint(s.z), __float_as_uint(s.w)};
        put<4>(static_cast<uint32_t*>(out) + p, v, nj - col, vec);
      }
    }
  }

  // Rows i0 .. of ni, columns j0 .. of nj, 16 rows at a time through LDS
  template <bool BF16>
  static constexpr int STORES = C::TB * 16 * (C::FT * (BF16 ? 2 : 4) / 16) / 64;

  template <bool BF16, bool WHOLE>
  __device__ __forceinline__ void store(char* lds, void* out, long long ld, int i0, int ni, int j0, int nj, int wf, int wt, bool vec) {
    constexpr int EB = BF16 ? 2 : 4, ROWB = C::FT * EB, NCH = ROWB / 16, RPP = 64 / NCH;
    const int tid = opaque(threadIdx.x), lane = tid & 63;
    char* mine = lds + C::STAGE + (tid >> 6) * (16 * C::FT * 4);
#pragma unroll
    for (int j = 0; j < C::TB; ++j) {
#pragma unroll
      for (int i = 0; i < C::FB; ++i) {
        const f32x4& v = acc[i][j];
        char* p = mine + stage_off<ROWB>(lane & 15, (i * 16 + 4 * (lane >> 4)) * EB);
        if constexpr (BF16) *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else *reinterpret_cast<float4*>(p) = float4{v[0], v[1], v[2], v[3]};
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const int c = lane % NCH, col = j0 + wf * C::FT + c * (16 / EB);
#pragma unroll
      for (int r0 = 0; r0 < 16; r0 += RPP) {
        const int r = r0 + lane / NCH, i = i0 + ((j >> 1) * C::WT + wt) * 32 + (j & 1) * 16 + r;
        using E = typename std::conditional<BF16, uint16_t, uint32_t>::type;
        E* dst = static_cast<E*>(out) + ((long long)i * ld + col);
        const char* src = mine + stage_off<ROWB>(r, c * 16);
        if constexpr (WHOLE) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        else if (r < 16 && i < ni && col < nj) put<16 / EB>(dst, reinterpret_cast<const E*>(src), nj - col, vec);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }

  // the stores that the wavefront issued, or 0 if it does not know
  __device__ __forceinline__ int write(char* lds, void* out, long long ld, int i0, int ni, int j0, int nj, int wf, int wt,
                                       bool bf16, bool vec) {
    if (vec && i0 + C::TM <= ni && j0 + C::TN <= nj) {
      if (bf16) return store<true, true>(lds, out, ld, i0, ni, j0, nj, wf, wt, true), STORES<true>;
      return store<false, true>(lds, out, ld, i0, ni, j0, nj, wf, wt, true), STORES<false>;
    }
    if (bf16) store<true, false>(lds, out, ld, i0, ni, j0, nj, wf, wt, vec);
    else store<false, false>(lds, out, ld, i0, ni, j0, nj, wf, wt, vec);
    return 0;
  }
};

// A tile of the call, and how much of k it adds up
struct Work {
  int i0, ni, j0, nc;
  char* out;
};

// Workgroups walk the tiles as the bf16 kernel's do.
template <class C>
__global__ void __launch_bounds__(C::THREADS, (C::THREADS / 256) * C::OCC) moe_gemm_mx(const GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  const int wave = uni((int)(threadIdx.x >> 6)), kw = C::KW == 1 ? 0 : wave;
  const int wf = C::KW == 1 ? wave % C::WF : 0, wt = C::KW == 1 ? wave / C::WF : 0;
  char* const ring = lds + kw * C::RING;
  const int tj = (a.n + C::TN - 1) / C::TN;
  const int oe = a.out_bf16 ? 2 : 4;
  const bool grouped = a.row_offset != nullptr;
  const GroupScan<C::TM> scan(a.row_offset, grouped ? a.L : 0, a.rows);
  const int ti = grouped ? scan.total : (a.rows + C::TM - 1) / C::TM;
  const int tiles = ti * tj, total = tiles * a.splits;
  TileM<C> g;

  auto start = [&](int b, Work& wk) {
    int tile = xcd_tile(b, total);
    if (tile >= total) return false;
    int s = 0, c0 = 0;
    if (a.splits > 1) {
      s = tile / tiles;
      tile -= s * tiles;
    }
    const int nc = split_range<C::KS>(a.k, a.splits, s, c0);
    int p, j;
    tile_at(tile, ti, tj, p, j);
    const Group gr = grouped ? scan.find(p) : Group{0, p, 0, a.rows, true};
    const int i0 = gr.m * C::TM, j0 = j * C::TN;
    g.fbase = static_cast<const char*>(a.w) + (long long)gr.e * a.es_w + (long long)j0 * a.ld_w + c0 / 2;
    g.tbase = static_cast<const char*>(a.x) + (long long)(gr.r0 + i0) * a.ld_x + (C::X4 ? c0 / 2 : c0);
    g.template offsets<C::FROW>(g.fv, a.ld_w, a.n - 1 - j0);
    g.template offsets<C::TROW>(g.tv, a.ld_x, gr.Me - 1 - i0);
    const char* ws = reinterpret_cast<const char*>(a.ws) + (long long)gr.e * a.es_ws + (long long)j0 * a.ld_ws + c0 / 32;
    const char* xs = reinterpret_cast<const char*>(a.xs) + (long long)(gr.r0 + i0) * a.ld_xs + c0 / 32;
#pragma unroll
    for (int i = 0; i < C::NSC; ++i) {
      const int q = g.scale_word(i), h = q / (C::TN + C::TM), r = q - h * (C::TN + C::TM);
      g.sp[i] = (r < C::TN ? ws + (long long)min(r, a.n - 1 - j0) * a.ld_ws : xs + (long long)min(r - C::TN, gr.Me - 1 - i0) * a.ld_xs) + 4 * h;
    }
    wk = Work{i0, gr.Me, j0, nc, static_cast<char*>(a.y) + ((long long)gr.r0 * a.ld_y + s * a.part) * oe};
    g.first(ring, nc, kw);
    return true;
  };

  Work cur, next;
  int b = blockIdx.x;
  int stores = 0;   // of the previous tile, possibly in flight
  bool more = start(b, cur), fresh = true;
  while (more) {
    g.multiply(ring, cur.ni - cur.i0, cur.nc, wf, wt, kw, stores, fresh);
    fresh = C::KW > 1;   // split wavefronts store before they copy
    stores = 0;
    b += gridDim.x;
    if constexpr (C::KW == 1) {
      lds_barrier();   // every wavefront is done with the ring
      more = start(b, next);
      stores = g.write(lds, cur.out, a.ld_y, cur.i0, cur.ni, cur.j0, a.n, wf, wt, a.out_bf16, a.vec_out);
    } else {
      g.store_split(lds, cur.out, a.ld_y, cur.i0, cur.ni, cur.j0, a.n, kw, a.out_bf16, a.vec_out);
      __syncthreads();   // the joined sums are read
      more = start(b, next);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    cur = next;
  }
}

//                        rows cols wavefronts ring spread workgroups per CU
template <bool X4> using Large = CfgM<X4, 256, 256, 2, 4, X4 ? 2 : 3, 4, 1>;
template <bool X4> using Wide = CfgM<X4, 192, 256, 2, 4, X4 ? 2 : 3, 4, 1>;
template <bool X4> using Medium = CfgM<X4, 128, 256, 2, 4, X4 ? 3 : 4, 4, 1>;
template <bool X4> using Square = CfgM<X4, 128, 128, 2, 2, X4 ? 2 : 3, 4, 2>;
template <bool X4> using Small = CfgM<X4, 64, 128, 1, 4, X4 ? 3 : 4, 4, 2>;
template <bool X4> using Split = CfgM<X4, 32, 32, 1, 1, X4 ? 2 : 3, 4, 1, 8>;
template <bool X4> using Split64 = CfgM<X4, 32, 64, 1, 1, X4 ? 3 : 4, 4, 1, 4>;
template <bool X4> using Deep = CfgM<X4, 128, 128, 2, 4, X4 ? 4 : 6, 4, 1>;
template <bool X4> using Few = CfgM<X4, 16, 32, 1, 1, X4 ? 3 : 4, 4, 1, 8>;
template <bool X4> using Thin = CfgM<X4, 32, 128, 1, 4, X4 ? 3 : 4, 4, X4 ? 2 : 3>;

template <class C>
hipError_t launch(const GemmArgs& a, hipStream_t s) {
  const long long nj = (a.n + C::TN - 1) / C::TN;
  const long long mi = a.row_offset ? ((long long)a.rows + (long long)a.L * (C::TM - 1)) / C::TM : (a.rows + C::TM - 1) / C::TM;
  const long long tiles = nj * mi * a.splits;
  if (tiles >= INT_MAX / 2) return launch_gemm_mx_any(a, s);   // the kernel counts tiles in int
  const long long grid = tiles > kCus ? kCus * C::OCC : (tiles + 7) / 8 * 8;
  moe_gemm_mx<C><<<(unsigned)grid, C::THREADS, 0, s>>>(a);
  return hipGetLastError();
}

template <bool X4>
hipError_t pick(int id, const GemmArgs& a, hipStream_t s) {
  switch (id) {
    case 1: return launch<Large<X4>>(a, s);
    case 2: return launch<Wide<X4>>(a, s);
    case 3: return launch<Medium<X4>>(a, s);
    case 4: return launch<Square<X4>>(a, s);
    case 5: return launch<Small<X4>>(a, s);
    case 6: return launch<Split<X4>>(a, s);
    case 7: return launch<Split64<X4>>(a, s);
    case 8: return launch<Deep<X4>>(a, s);
    case 9: return launch<Few<X4>>(a, s);
    case 10: return launch<Thin<X4>>(a, s);
  }
  return hipErrorInvalidValue;
}

template <class C>
constexpr GemmTile timed(double a, double c, double b, double o, bool once = false) {
  return GemmTile{C::TM, C::TN, C::OCC, C::KW, a, c, b, o, once};
}

}  // namespace

const GemmTile kMxTiles[2][kMxGemmTiles] = {
    {timed<Large<false>>(0.73, 1.0, 1.0, 6), timed<Wide<false>>(0.68, 0.8, 0.8, 5), timed<Medium<false>>(0.50, 0.6, 0.6, 5),
     timed<Square<false>>(0.37, 0.5, 0.4, 4), timed<Small<false>>(0.28, 0.42, 0.25, 4), timed<Split<false>>(0.6, 0.6, 0.6, 2),
     timed<Split64<false>>(0.60, 0.6, 0.6, 2), timed<Deep<false>>(0.37, 0.4, 0.4, 5, true), timed<Few<false>>(0.50, 0.55, 0.55, 2),
     timed<Thin<false>>(0.28, 0.3, 0.2, 3)},
    {timed<Large<true>>(0.73, 1.0, 1.0, 6), timed<Wide<true>>(0.68, 0.8, 0.8, 5), timed<Medium<true>>(0.50, 0.6, 0.6, 5),
     timed<Square<true>>(0.37, 0.5, 0.4, 4), timed<Small<true>>(0.28, 0.42, 0.25, 4), timed<Split<true>>(0.6, 0.6, 0.6, 2),
     timed<Split64<true>>(0.60, 0.6, 0.6, 2), timed<Deep<true>>(0.37, 0.4, 0.4, 5, true), timed<Few<true>>(0.50, 0.55, 0.55, 2),
     timed<Thin<true>>(0.28, 0.3, 0.2, 3)}};

hipError_t launch_gemm_mx(int id, const GemmArgs& a, hipStream_t s) { return a.x_e2m1 ? pick<true>(id, a, s) : pick<false>(id, a, s); }

}  // namespace moe
