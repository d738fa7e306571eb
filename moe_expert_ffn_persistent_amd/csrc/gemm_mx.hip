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
// or 256 k of e2m1 beside 128-byte ones (two MFMAs a 16 x 16 block). An NS-deep LDS
// ring is filled by direct-to-LDS copies between the MFMAs of an earlier stage. A
// ragged last stage is zeros in LDS, with scales of 1.
//
// Scales come in groups of 512 k, 16 bytes of every row, into buffers of their own: a
// copy then touches 16 rows. Copied with each stage, 128 k of 64 rows at a time,
// their scattered lines were the kernel's bound (8192 x 7168 x 4096 e4m3 203 us
// where the same copies from one line took 169, e2m1 145 and 108).
#include <type_traits>
#include <utility>

#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

// 16 (or 4) bytes a lane from base + voff (bytes) to LDS m0 + 16 (4) * lane; s_nop: m0's
// wait state (see dma16 in ffn_common.hpp), and the 5 after a base that a lane read wrote
// (where there are more bases than registers they are read back right before)
__device__ __forceinline__ void dma16s(uint32_t voff, const char* base, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(m0) : "memory", "m0");
}
__device__ __forceinline__ void dma4s(uint32_t voff, const char* base, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "s"(m0) : "memory", "m0");
}

// f(0) .. f(N - 1), the numbers as types: whole loops of what is chosen at compile
// time (an unrolled loop of this size is left rolled, and its arrays go to memory)
template <class F, int... I>
__device__ __forceinline__ void each_of(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

// KW > 1: KW wavefronts split the sum, a run of stages each: a ring each, sums
// joined in LDS.
template <bool X4_, int M_, int TM_, int TN_, int WT_, int WF_, int NS_, int SP_, int OCC_, int GW_, int KW_ = 1>
struct CfgM {
  static constexpr bool X4 = X4_;
  static constexpr int TM = TM_, TN = TN_, WT = WT_, WF = WF_, NS = NS_, SP = SP_, OCC = OCC_;
  static constexpr int KW = KW_, NW = WT * WF, THREADS = 64 * NW * KW;
  static constexpr int KS = M_ * (X4 ? 256 : 128), H = KS / 128;   // k of a stage, MFMAs of a block in it
  static constexpr int FROW = KS / 2, TROW = X4 ? FROW : KS;       // bytes of a row in a stage
  static constexpr int TT = TM / WT, FT = TN / WF;
  static constexpr int TB = TT / 16, FB = FT / 16, NB = TB * FB;   // 16 x 16 blocks of a wavefront
  static constexpr int TP = TB > 1 ? TB / 2 : 1;                   // 32-row blocks
  static constexpr int NIT = TM * TROW / 1024 / NW, NIF = TN * FROW / 1024 / NW;
  static constexpr int NI = NIT + NIF;
  static constexpr int F_BYTES = TN * FROW, T_BYTES = TM * TROW;
  static constexpr int STAGE = F_BYTES + T_BYTES;
  static constexpr int EPI = NW * 16 * FT * 4;
  static constexpr int RING = NS * STAGE;
  // Scales: a group is GW words of every row, SPG stages; RB copies of CR rows
  // (weights' first), NG of them a wavefront's. Group G's buffer is free once group
  // G - NBUF has been multiplied, and its copies land by stage G SPG if they go out
  // with that stage's or earlier ones: with the SL stages up to it, PP copies each.
  static constexpr int GW = GW_, SPG = GW * 128 / KS, NBUF = NS - 1 <= SPG ? 2 : 3;
  static constexpr int CR = 64 / GW, RB = (TN + TM) / CR, NG = (RB + NW - 1) / NW, GROUP = RB * 256;
  static constexpr int SL0 = (NBUF - 1) * SPG - NS + 2, SL = SL0 < SPG ? SL0 : SPG, PP = (NG + SL - 1) / SL;
  static constexpr int WAVES_LDS = RING + NBUF * GROUP;   // of the wavefronts that share a ring
  static constexpr int LDS = KW * WAVES_LDS;
  static_assert(SL >= 1 && TN % CR == 0 && TM % CR == 0 && 64 % GW == 0, "scale groups");
  static_assert(RING - STAGE >= EPI || KW > 1, "the epilogue stages behind the next tile's first stage");
  static_assert(KW == 1 || (NW == 1 && TM <= 32), "split wavefronts hold the whole tile each");
  static_assert(KW == 1 || RING >= TM * TN * 4, "a wavefront's sums fit its ring");
  // register sets of fragments: of rows, read BUF - 1 blocks ahead, and of weights
  static constexpr int BUF = X4 ? 4 : 2, WBUF = H > 1 ? 2 : 1;
  // copies of a stage when only ntp 32-row blocks a wavefront hold rows
  static constexpr int copies(int ntp) { return NIF + NIT * ntp / TP; }
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
  else if constexpr (ROW == 128) return c ^ ((r >> 1) & 7);
  else return c ^ (r & 15);
}
template <int ROW>
__device__ __forceinline__ int chunk_in(int r, int p) {
  if constexpr (ROW == 64) {
    const int x = p ^ ((r >> 2) & 3);
    return x ^ ((x & 1) << 1);
  } else {
    return chunk_at<ROW>(r, p);
  }
}

template <class C, bool EVEN>
struct TileM {
  const char *fbase, *tbase, *wsbase, *xsbase;
  uint32_t fv[C::NIF], tv[C::NIT];
  uint32_t sv[C::NG];       // this lane's scale word in group 0
  int k;                    // what is added up
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

  // copy i of stage kt
  template <int i>
  __device__ __forceinline__ void issue(int kt, uint32_t slot) const {
    const uint32_t wave = wave_of();
    slot = uni(slot);
    if constexpr (i < C::NIF) dma16s(fv[i], fbase + (long long)kt * C::FROW, slot + (wave + C::NW * i) * 1024);
    else dma16s(tv[i - C::NIF], tbase + (long long)kt * C::TROW, slot + C::F_BYTES + (wave + C::NW * (i - C::NIF)) * 1024);
  }

  // Scale copy i of a wavefront is copy b of the group, rows CR b ..: lane l has word
  // l % GW of row l / GW
  __device__ __forceinline__ static int copy_of(int i) { return i * C::NW + wave_of(); }
  __device__ __forceinline__ const char* scales_of(int b, int group) const { return (b < C::TN / C::CR ? wsbase : xsbase) + group * (4ll * C::GW); }
  __device__ __forceinline__ static uint32_t buffer(int group) { return C::RING + (C::NBUF == 2 ? group & 1 : group % C::NBUF) * C::GROUP; }

  // words that hold four scales of the sum (the others: issue_tail)
  template <int i>
  __device__ __forceinline__ void issue_group(int group, uint32_t lds) const {
    const int b = copy_of(i);
    if (C::RB % C::NW != 0 && b >= C::RB) return;
    const uint32_t dst = uni(lds + buffer(group) + b * 256);
    if ((group + 1) * C::GW <= k / 128 || group * C::GW + (int)threadIdx.x % C::GW < k / 128) dma4s(sv[i], scales_of(b, group), dst);
  }

  // the scale copies that go out with stage t > 0
  __device__ __forceinline__ void issue_scales(int t, uint32_t lds) const {
    const int group = (t + C::SPG - 1) / C::SPG, p = t - group * C::SPG + C::SL - 1;
    if (p < 0 || group * (C::GW * 128) >= k) return;
    each<C::SL>([&](auto s) {
      if (p == s)
        each<C::PP>([&](auto i) {
          if constexpr (s * C::PP + i < C::NG) issue_group<s * C::PP + i>(group, lds);
        });
    });
  }

  // 16 bytes at `src` of which `n` e4m3 bytes (PACKED: e2m1 codes) exist; a short loop,
  // since a longer body slows every short call by its size (unrolled over words: 1 x 7170
  // x 4096 8.6 to 9.6 us)
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

  template <int copy>
  __device__ __forceinline__ void tail_copy(int kt, int left, char* slot) const {
    constexpr bool W = copy < C::NIF, PACKED = W || C::X4;
    constexpr int i = W ? copy : copy - C::NIF, E = PACKED ? 32 : 16;   // elements of 16 bytes
    int r, c;
    place<W ? C::FROW : C::TROW>(i, r, c);
    const int have = left - c * E;
    if (have >= E) {
      issue<copy>(kt, (uint32_t)(uintptr_t)slot);
    } else {
      const char* src = W ? fbase + (long long)kt * C::FROW + fv[W ? i : 0] : tbase + (long long)kt * C::TROW + tv[W ? 0 : i];
      char* at = slot + (W ? 0 : C::F_BYTES) + (wave_of() + C::NW * i) * 1024 + (threadIdx.x & 63) * 16;
      *reinterpret_cast<uint4*>(at) = have > 0 ? partial<PACKED>(src, have) : uint4{0, 0, 0, 0};
    }
  }

  // the last stage when it holds only `left` < KS k
  __device__ __forceinline__ void issue_tail(int kt, int left, char* lds) const {
    char* const slot = lds + kt % C::NS * C::STAGE;
    each<C::NI>([&](auto i) { tail_copy<i>(kt, left, slot); });
    // the stage's scale words that are not whole: 1 for blocks that are not there
    // (what lies behind the row may be NaN)
    const int group = kt / C::SPG, w = group * C::GW + (int)threadIdx.x % C::GW;
    if (w >= k / 128 && w < (kt + 1) * C::H) {
#pragma unroll
      for (int i = 0; i < C::NG; ++i) {
        const int b = copy_of(i);
        if (C::RB % C::NW != 0 && b >= C::RB) continue;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(scales_of(b, group)) + sv[i];
        uint32_t word = 0x7f7f7f7fu;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (w * 128 + j * 32 < k) word = (word & ~(0xffu << (8 * j))) | (uint32_t)src[j] << (8 * j);
        *reinterpret_cast<uint32_t*>(lds + buffer(group) + b * 256 + (threadIdx.x & 63) * 4) = word;
      }
    }
  }

  // e2m1 fragments are half of the instruction's operand
  using Rows = typename std::conditional<C::X4, i32x4, i32x8>::type;
  struct Frags {
    i32x4 a[C::WBUF][C::FB];
    Rows b[C::BUF];
    int sa[C::WBUF][C::FB], sb[C::BUF];
  };
  // Where a wavefront reads a stage: its bases, and the lane's bytes in them
  struct View {
    const char *w, *x;
    const uint8_t* s;
  };
  __device__ __forceinline__ static View view(const char* lds, int kt, const char* stage, int wf, int wt) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    return View{stage + (wf * C::FT + r16) * C::FROW, stage + C::F_BYTES + (wt * 32 + r16) * C::TROW,
                reinterpret_cast<const uint8_t*>(lds) + buffer(kt / C::SPG) + kt % C::SPG * (4 * C::H) + r16 * (4 * C::GW) + q};
  }

  // Weight fragment i of 128 k number h. Rows are 16 apart, so the lane's place in
  // them is chunk_at of its own row.
  template <int i, int h, int buf>
  __device__ __forceinline__ static void load_w(Frags& f, const View& v, int wf) {
    const int r16 = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
    const uint4 w = *reinterpret_cast<const uint4*>(v.w + i * 16 * C::FROW + (chunk_at<C::FROW>(r16, 4 * h + q) << 4));
    f.a[buf][i] = i32x4{(int)w.x, (int)w.y, (int)w.z, (int)w.w};
    f.sa[buf][i] = v.s[(wf * C::FT + i * 16) * (4 * C::GW) + 4 * h];
  }
  // Fragment of 16-row block j, 128 k number h. e4m3: elements 16 q .. and 64 + 16 q
  // .., which meet the weights' 32 q .. (operand placement: gemm_mx_any.hip). 32-row
  // blocks go to the row wavefronts in turn.
  template <int j, int h, int buf>
  __device__ __forceinline__ static void load_x(Frags& f, const View& v, int wt) {
    constexpr int row = (j >> 1) * C::WT * 32 + (j & 1) * 16;
    const int r16 = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
    const char* p = v.x + row * C::TROW;
    const uint4 lo = *reinterpret_cast<const uint4*>(p + (chunk_at<C::TROW>(r16, (C::X4 ? 4 : 8) * h + q) << 4));
    if constexpr (C::X4) {
      f.b[buf] = i32x4{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w};
    } else {
      const uint4 hi = *reinterpret_cast<const uint4*>(p + (chunk_at<C::TROW>(r16, 8 * h + 4 + q) << 4));
      f.b[buf] = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    }
    f.sb[buf] = v.s[(C::TN + wt * 32 + row) * (4 * C::GW) + 4 * h];
  }

  __device__ __forceinline__ static i32x8 operand(const i32x4& v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
  __device__ __forceinline__ static i32x8 operand(const i32x8& v) { return v; }

  // One stage. Only the first NTP of the wavefront's 32-row blocks are multiplied.
  template <bool COPY, int NTP>
  __device__ __forceinline__ void compute(const char* lds, int kt, const char* stage, int wf, int wt, uint32_t slot) {
    constexpr int TB = C::TB == 1 ? 1 : 2 * NTP, NB = C::H * TB, NI = C::copies(NTP);   // NB blocks of rows
    const View v = view(lds, kt, stage, wf, wt);
    Frags f;
    load_x<0, 0, 0>(f, v, wt);
    load_w<0, 0, 0>(f, v, wf);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (COPY) issue_scales(kt + C::NS - 1, (uint32_t)(uintptr_t)lds);
    each<NB * C::FB>([&](auto b) {
      constexpr int jj = b / C::FB, j = jj % TB, h = jj / TB, i = b % C::FB;
      // the first block's MFMAs: the rest of the weights, and the blocks ahead
      if constexpr (b + 1 < C::FB) load_w<b + 1, 0, 0>(f, v, wf);
      constexpr int ahead = jj == 0 ? (b + 1 < C::BUF ? b + 1 : NB) : i == 0 ? jj + C::BUF - 1 : NB;
      if constexpr (ahead < NB) load_x<ahead % TB, ahead / TB, ahead % C::BUF>(f, v, wt);
      if constexpr (jj == 0 && i == C::FB - 1)   // fewer MFMAs than blocks ahead
        each<(C::BUF - 1 > C::FB ? C::BUF - 1 - C::FB : 0)>([&](auto e) {
          constexpr int more = C::FB + 1 + e;
          if constexpr (more < NB) load_x<more % TB, more / TB, more % C::BUF>(f, v, wt);
        });
      // the next 128 k's weights, into the set that the one before left
      if constexpr (h + 1 < C::H && (TB == 1 ? j == 0 : j == 1)) load_w<i, (h + 1) % C::H, (h + 1) % 2>(f, v, wf);
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(f.a[h % C::WBUF][i]), operand(f.b[jj % C::BUF]), acc[i][j], 4,
                                                                   C::X4 ? 4 : 0, 0, f.sa[h % C::WBUF][i], 0, f.sb[jj % C::BUF]);
      if constexpr (COPY)
        each<NI>([&](auto c) {
          if constexpr (C::issue_slot(c, NB * C::FB, NI) == b) issue<c>(kt + C::NS - 1, slot);
        });
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  // Copies of the first stage, and of the first group of scales
  __device__ __forceinline__ void first(char* lds) const {
    if (k == 0) return;
    each<C::NG>([&](auto i) { issue_group<i>(0, (uint32_t)(uintptr_t)lds); });
    if (k >= C::KS) {
      each<C::NI>([&](auto i) { issue<i>(0, (uint32_t)(uintptr_t)lds); });
    } else if constexpr (!EVEN) {
      issue_tail(0, k, lds);
    }
  }

  // All of k, the first stage's copies already issued
  template <int NTP>
  __device__ __forceinline__ void mainloop(char* lds, int wf, int wt, int stores, bool fresh) {
    constexpr int NI = C::copies(NTP);
#pragma unroll
    for (int i = 0; i < C::FB; ++i)
#pragma unroll
      for (int j = 0; j < C::TB; ++j) acc[i][j] = f32x4{};
    const uint32_t ring = (uint32_t)(uintptr_t)lds;
    const int full = k / C::KS, left = EVEN ? 0 : k % C::KS, nk = full + (left != 0);
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
        if (s < nk) issue_scales(s, ring);
        if (s < full) {
          each<NI>([&](auto i) { issue<i>(s, ring + s * C::STAGE); });
        } else if constexpr (!EVEN) {
          if (s < nk) issue_tail(s, left, lds);
        }
      }
    }
    int slot = 0;
    const int nmain = full - (C::NS - 1);
    for (int s = 0; s < nmain; ++s) {
      // the stage has landed; of later ones this many copies at least are behind it
      // (the scales' stand before their stage's and are not counted)
      if (s || fresh) vm_wait<NI * (C::NS - 2)>();
      if constexpr (C::KW == 1) lds_barrier();
      const int nslot = slot == 0 ? C::NS - 1 : slot - 1;
      compute<true, NTP>(lds, s, lds + slot * C::STAGE, wf, wt, ring + nslot * C::STAGE);
      slot = slot + 1 == C::NS ? 0 : slot + 1;
    }
    for (int s = max(nmain, 0); s < nk; ++s) {
      if (s == 0 && !fresh) {
      } else if (left) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      else vm_wait_ahead<NI, C::NS - 2>(nk - 1 - s);
      if constexpr (C::KW == 1) lds_barrier();
      if constexpr (!EVEN) {
        if (left && s + C::NS - 1 == full) {
          issue_scales(full, ring);
          issue_tail(full, left, lds);
        }
      }
      compute<false, NTP>(lds, s, lds + slot * C::STAGE, wf, wt, 0);
      slot = slot + 1 == C::NS ? 0 : slot + 1;
    }
  }

  // The tile's `rows` rows (at least one)
  __device__ __forceinline__ void multiply(char* lds, int rows, int wf, int wt, int stores, bool fresh) {
    const int blocks = (min(rows, C::TM) + 32 * C::WT - 1) / (32 * C::WT);
    if constexpr (C::TB >= 4) {
      if (blocks == 1) return mainloop<1>(lds, wf, wt, stores, fresh);
    }
    if constexpr (C::TB >= 6) {
      if (blocks == 2) return mainloop<2>(lds, wf, wt, stores, fresh);
    }
    if constexpr (C::TB >= 8) {
      if (blocks == 3) return mainloop<3>(lds, wf, wt, stores, fresh);
    }
    mainloop<C::TP>(lds, wf, wt, stores, fresh);
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
    char* mine = lds + kw * C::WAVES_LDS;
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
        const float4 o = *reinterpret_cast<const float4*>(lds + w * C::WAVES_LDS + stage_off<ROWB>(r, c * 16));
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

// An address alike for the wavefront, in scalar registers
__device__ __forceinline__ const char* uni_ptr(const char* p) {
  const uint64_t v = (uint64_t)p;
  return reinterpret_cast<const char*>((uint64_t)(uint32_t)uni((int)v) | (uint64_t)(uint32_t)uni((int)(v >> 32)) << 32);
}

// A tile of the call
struct Work {
  int i0, ni, j0;
  char* out;
};

// Workgroups walk the tiles as the bf16 kernel's do. EVEN: the sum is whole stages
// long; short calls take longer by the size of the code that ends it otherwise (1 x 7168
// x 4096 W4A8: 5 KB 6.5 us, 18 KB 7.5), so it is built for tiles of few rows.
template <class C, bool EVEN>
__global__ void __launch_bounds__(C::THREADS, (C::THREADS / 256) * C::OCC) moe_gemm_mx(const GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  const int wave = uni((int)(threadIdx.x >> 6)), kw = C::KW == 1 ? 0 : wave;
  const int wf = C::KW == 1 ? wave % C::WF : 0, wt = C::KW == 1 ? wave / C::WF : 0;
  char* const ring = lds + kw * C::WAVES_LDS;
  const int tj = (a.n + C::TN - 1) / C::TN;
  const int oe = a.out_bf16 ? 2 : 4;
  const bool grouped = a.row_offset != nullptr;
  const GroupScan<C::TM> scan(a.row_offset, grouped ? a.L : 0, a.rows);
  const int ti = grouped ? scan.total : (a.rows + C::TM - 1) / C::TM;
  const int tiles = ti * tj, total = tiles * a.splits;
  TileM<C, EVEN> g;

  auto start = [&](int b, Work& wk) {
    int tile = xcd_tile(b, total);
    if (tile >= total) return false;
    int s = 0, c0 = 0;
    if (a.splits > 1) {
      s = tile / tiles;
      tile -= s * tiles;
    }
    int nc = split_range<C::KS>(a.k, a.splits, s, c0);
    if constexpr (C::KW > 1) {   // this wavefront's share: whole stages, the first ones have one more
      const int all = (nc + C::KS - 1) / C::KS, each = all / C::KW, more = all - each * C::KW;
      const int from = (kw * each + min(kw, more)) * C::KS;
      c0 += from;
      nc = max(0, min(nc - from, (each + (kw < more)) * C::KS));
    }
    int p, j;
    tile_at(tile, ti, tj, p, j);
    const Group gr = grouped ? scan.find(p) : Group{0, p, 0, a.rows, true};
    const int i0 = gr.m * C::TM, j0 = j * C::TN;
    g.k = uni(nc);
    g.fbase = uni_ptr(static_cast<const char*>(a.w) + (long long)gr.e * a.es_w + (long long)j0 * a.ld_w + c0 / 2);
    g.tbase = uni_ptr(static_cast<const char*>(a.x) + (long long)(gr.r0 + i0) * a.ld_x + (C::X4 ? c0 / 2 : c0));
    g.template offsets<C::FROW>(g.fv, a.ld_w, a.n - 1 - j0);
    g.template offsets<C::TROW>(g.tv, a.ld_x, gr.Me - 1 - i0);
    g.wsbase = uni_ptr(reinterpret_cast<const char*>(a.ws) + (long long)gr.e * a.es_ws + (long long)j0 * a.ld_ws + c0 / 32);
    g.xsbase = uni_ptr(reinterpret_cast<const char*>(a.xs) + (long long)(gr.r0 + i0) * a.ld_xs + c0 / 32);
#pragma unroll
    for (int i = 0; i < C::NG; ++i) {
      const int rb = g.copy_of(i), r = rb * C::CR + (int)(threadIdx.x & 63) / C::GW;
      const int row = r < C::TN ? min(r, a.n - 1 - j0) : min(r - C::TN, gr.Me - 1 - i0);
      g.sv[i] = (uint32_t)row * (uint32_t)(r < C::TN ? a.ld_ws : a.ld_xs) + threadIdx.x % C::GW * 4;
    }
    wk = Work{i0, gr.Me, j0, static_cast<char*>(a.y) + ((long long)gr.r0 * a.ld_y + s * a.part) * oe};
    g.first(ring);
    return true;
  };

  Work cur;
  int b = blockIdx.x;
  if constexpr (C::KW > 1) {   // the next tile's copies wait for the stores: the rings hold the sums
    for (; start(b, cur); b += gridDim.x) {
      g.multiply(ring, cur.ni - cur.i0, wf, wt, 0, true);
      g.store_split(lds, cur.out, a.ld_y, cur.i0, cur.ni, cur.j0, a.n, kw, a.out_bf16, a.vec_out);
      __syncthreads();   // the joined sums are read
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  } else {
    Work next;
    int stores = 0;   // of the previous tile, possibly in flight
    bool more = start(b, cur), fresh = true;
    while (more) {
      g.multiply(ring, cur.ni - cur.i0, wf, wt, stores, fresh);
      fresh = false;
      b += gridDim.x;
      lds_barrier();   // every wavefront is done with the ring
      more = start(b, next);
      stores = g.write(lds, cur.out, a.ld_y, cur.i0, cur.ni, cur.j0, a.n, wf, wt, a.out_bf16, a.vec_out);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      cur = next;
    }
  }
}

// 128 (e2m1: 256) k a stage, or twice that; rows, columns; wavefronts along them; ring; spread; workgroups a
// compute unit; scale words a group; wavefronts that split the sum.
// Stages of 128-byte weight rows stream weights best (e4m3 rows, 32 experts x 128
// rows, 7168 to 4096: 94 us in 64-byte pieces, 87 so), where LDS has room for them.
template <bool X4> using Large = CfgM<X4, 1, 256, 256, 2, 4, X4 ? 2 : 3, 4, 1, 4>;
template <bool X4> using Wide = CfgM<X4, 1, 192, 256, 2, 4, X4 ? 2 : 3, 4, 1, X4 ? 8 : 4>;
template <bool X4> using Medium = CfgM<X4, 1, 128, 256, 2, 4, X4 ? 3 : 4, 4, 1, 4>;
using Small = CfgM<true, 1, 64, 128, 1, 4, 3, 4, 2, 4>;                            // of e2m1 rows only
template <bool X4> using Deep = CfgM<X4, 2, 128, 128, 2, 4, 2, 4, 1, 4>;           // for calls that give no compute unit a second tile
using Split = CfgM<false, 1, 32, 32, 1, 1, 3, 4, 1, 4, 8>;                         // of e4m3 rows only
template <bool X4> using Split64 = CfgM<X4, 1, 32, 64, 1, 1, X4 ? 3 : 4, 4, 1, 4, 4>;
template <bool X4> using Few = CfgM<X4, X4 ? 1 : 2, 16, 32, 1, 1, X4 ? 3 : 2, 4, 1, 4, 8>;
template <bool X4> using Thin = CfgM<X4, X4 ? 1 : 2, 32, 128, 1, 4, 3, 4, 2, 4>;
using Thin16 = CfgM<false, 2, 16, 128, 1, 4, 3, 4, 2, 4>;                          // of e4m3 rows only

template <class C>
hipError_t launch(const GemmArgs& a, hipStream_t s) {
  const long long tiles = gemm_tiles(a, C::TM, C::TN);
  if (tiles >= kMostTiles) return launch_gemm_mx_any(a, s);   // only whole sums (ops_api.cpp)
  const long long grid = tiles > kCus ? kCus * C::OCC : (tiles + 7) / 8 * 8;
  if constexpr (C::TM <= 32) {
    if (a.k % C::KS == 0) {
      moe_gemm_mx<C, true><<<(unsigned)grid, C::THREADS, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  moe_gemm_mx<C, false><<<(unsigned)grid, C::THREADS, 0, s>>>(a);
  return hipGetLastError();
}

template <bool X4>
hipError_t pick(int id, const GemmArgs& a, hipStream_t s) {
  switch (id) {
    case 1: return launch<Large<X4>>(a, s);
    case 2: return launch<Wide<X4>>(a, s);
    case 3: return launch<Medium<X4>>(a, s);
    case 4:
      if constexpr (X4) return launch<Small>(a, s);
      break;
    case 5: return launch<Deep<X4>>(a, s);
    case 6:
      if constexpr (!X4) return launch<Split>(a, s);
      break;
    case 7: return launch<Split64<X4>>(a, s);
    case 8: return launch<Few<X4>>(a, s);
    case 9: return launch<Thin<X4>>(a, s);
    case 10:
      if constexpr (!X4) return launch<Thin16>(a, s);
  }
  return hipErrorInvalidValue;
}

template <class C>
constexpr GemmTile timed(double a, double c, double b, double o, bool once = false) {
  return GemmTile{C::TM, C::TN, C::OCC, C::KW, a, c, b, o, once};
}

}  // namespace

const GemmTile kMxTiles[2][kMxGemmTiles] = {
    {timed<Large<false>>(0.36, 1.33, 1.33, 7.1), timed<Wide<false>>(0.47, 1.05, 1.05, 6.4), timed<Medium<false>>(0.49, 0.74, 0.74, 5.9),
     GemmTile{}, timed<Deep<false>>(0.31, 0.43, 0.43, 5.0, true), timed<Split>(0.405, 0.405, 0.405, 4.03),
     timed<Split64<false>>(0.45, 0.45, 0.45, 4.09), timed<Few<false>>(0.214, 0.214, 0.214, 4.17), timed<Thin<false>>(0.177, 0.25, 0.206, 4.37),
     timed<Thin16>(0.169, 0.20, 0.134, 4.08)},
    {timed<Large<true>>(0.55, 1.89, 1.89, 6.6), timed<Wide<true>>(0.73, 1.51, 1.51, 6.1), timed<Medium<true>>(0.58, 1.08, 1.08, 5.6),
     timed<Small>(0.31, 0.44, 0.36, 4.76), timed<Deep<true>>(0.29, 0.55, 0.55, 5.5, true), GemmTile{},
     timed<Split64<true>>(0.59, 0.59, 0.59, 4.1), timed<Few<true>>(0.455, 0.455, 0.455, 4.1), timed<Thin<true>>(0.33, 0.50, 0.26, 4.4),
     GemmTile{}}};

hipError_t launch_gemm_mx(int id, const GemmArgs& a, hipStream_t s) { return a.x_e2m1 ? pick<true>(id, a, s) : pick<false>(id, a, s); }

}  // namespace moe
