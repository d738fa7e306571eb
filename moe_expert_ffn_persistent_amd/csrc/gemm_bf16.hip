// Grouped bf16 matrix products (forward, input gradient, weight gradient) for
// 16-byte aligned operands:
//
//   out(i, j) = sum over c of T(i, c) F(j, c)
//   forward  i = row, j = n, c = k     T = x            F = W[e]
//   dgrad    i = row, j = k, c = n     T = dy           F = W[e]^T
//   wgrad    i = n,   j = k, c = row   T = dy^T         F = x^T
//
// F is the MFMA's A operand and T its B operand (v_mfma_f32_32x32x16_bf16), so
// a lane ends up with one output row i and runs of four consecutive columns j.
// An operand whose unit stride is c is staged in LDS as rows of 64 c (128
// bytes) and read 16 bytes a lane; one whose unit stride is i or j (marked TR)
// is staged as it lies in memory, 64 rows of c, and read by
// ds_read_b64_tr_b16, which hands each lane four consecutive c of its column.
// No operand is transposed through registers or in HBM.
//
// A stage is 64 c wide; an NS-deep ring of stages is filled by direct-to-LDS
// copies issued between the MFMAs of an earlier stage, one workgroup barrier
// per stage. A ragged end (the last c of a row, or of an expert's rows in
// wgrad) is zeros in LDS: lanes past the end write a zero instead of copying.
// Rows i past an expert's end repeat its last row and are not stored.
#include <climits>

#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

// LDS byte addresses are the low words of the generic pointers used here
#pragma clang diagnostic ignored "-Wint-to-pointer-cast"

constexpr int kBK = 64;   // c per stage

typedef short s16x4 __attribute__((ext_vector_type(4)));

// 16 bytes a lane from base + voff (bytes) to LDS m0 + 16 * lane;
// s_nop: m0's wait state (see dma16 in ffn_common.hpp)
__device__ __forceinline__ void dma16s(uint32_t voff, const char* base, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(m0) : "memory", "m0");
}

// KW > 1: the workgroup's KW wavefronts share one small tile and split c: each
// takes every KW-th stage through a ring of its own, without barriers, and
// their sums are joined in LDS in wavefront order. For calls with few tiles,
// where one wavefront's chain of stages would leave the memory idle.
template <int TM_, int TN_, int WT_, int WF_, int NS_, int SP_, int OCC_, int KW_ = 1>
struct CfgG {
  static constexpr int TM = TM_, TN = TN_, WT = WT_, WF = WF_, NS = NS_, SP = SP_;
  static constexpr int OCC = OCC_;                 // workgroups per CU that LDS and registers are cut for
  static constexpr int KW = KW_;
  static constexpr int NW = WT * WF, THREADS = 64 * NW * KW;
  static constexpr int TT = TM / WT, FT = TN / WF; // rows and columns of a wavefront
  static constexpr int TB = TT > 32 ? TT / 32 : 1, FB = FT / 32;   // 16 rows fill half a block
  static constexpr int T_BYTES = TM * kBK * 2, F_BYTES = TN * kBK * 2;
  static constexpr int STAGE = T_BYTES + F_BYTES;
  static constexpr int NIT = T_BYTES / 1024 / NW, NIF = F_BYTES / 1024 / NW, NI = NIT + NIF;
  static constexpr int EPI = NW * 32 * FT * 4;     // epilogue staging: 32 rows a wavefront, fp32
  static constexpr int RING = NS * STAGE;
  // the epilogue stages behind the next tile's first stage
  static constexpr int LDS = KW > 1 || RING >= STAGE + EPI ? KW * RING : STAGE + EPI;
  static_assert(KW == 1 || (NW == 1 && TM <= 32), "split wavefronts hold the whole tile each");
  static constexpr int issue_slot(int i, int nm) { return i * nm * SP / (NI * 8); }
  static_assert(T_BYTES % (1024 * NW) == 0 && F_BYTES % (1024 * NW) == 0, "copies split evenly over the wavefronts");
  static_assert(NS >= 2 && NI * (NS - 1) <= 63, "vmcnt range");
  static_assert(LDS * OCC <= 160 * 1024, "LDS");
};

// One operand: TX rows (i or j) by 64 c a stage.
template <bool TR, int TX, int NW>
struct Operand {
  __device__ __forceinline__ static int wave_of() { return NW == 1 ? 0 : uni((int)(threadIdx.x >> 6)); }
  static constexpr int NI = TX * kBK * 2 / 1024 / NW;   // 1 KiB copies of a wavefront per stage
  static constexpr int RB = TR ? TX * 2 : kBK * 2;      // bytes of an LDS row
  static constexpr int RPI = 1024 / RB;                 // LDS rows per copy
  static_assert(1024 % RB == 0, "a copy fills whole LDS rows");
  const char* base;        // stage 0 (uniform)
  long long step;          // bytes from one stage to the next
  long long istep;         // TR: bytes between this wavefront's copies
  uint32_t voff[TR ? 1 : NI];

  // Physical place of what a lane reads. Normal rows: chunk c of row r sits at
  // c ^ (r >> 1 & 7), so that 16 rows at one chunk hit distinct banks.
  // TR rows: a transposing read takes 64 bytes of four consecutive rows for 32
  // lanes, so 64-byte pieces are spread by the row over the 256-byte bank line.
  __device__ __forceinline__ static int swz(int r) {
    constexpr int NG = RB / 64;
    if constexpr (!TR) return (r >> 1) & 7;
    else if constexpr (NG >= 4) return r & 3;
    else if constexpr (NG == 2) return (r >> 1) & 1;
    else return 0;
  }

  // p: element (row 0, c 0) of the tile's matrix; x0: the tile's first row (i
  // or j) of `nx`; ld: elements between rows of memory
  __device__ __forceinline__ void setup(const void* p, long long ld, int x0, int nx) {
    const int wave = wave_of(), lane = threadIdx.x & 63;
    const char* b = static_cast<const char*>(p);
    if constexpr (!TR) {
      base = b + (long long)x0 * ld * 2;
      step = kBK * 2;
      istep = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = (wave + NW * i) * RPI + lane / 8;
        const int c = (lane & 7) ^ swz(r);
        voff[i] = (uint32_t)min(r, nx - 1 - x0) * (uint32_t)(ld * 2) + c * 16;
      }
    } else {
      const int r = lane * 16 / RB, pc = (lane * 16 % RB) / 16;
      const int c = pc ^ (swz(wave * RPI + r) << 2);   // logical 16-byte piece
      base = b + (long long)wave * RPI * ld * 2;
      step = (long long)kBK * ld * 2;
      istep = (long long)NW * RPI * ld * 2;
      voff[0] = (uint32_t)r * (uint32_t)(ld * 2) + (uint32_t)min(x0 + c * 8, nx - 8) * 2;
    }
  }

  __device__ __forceinline__ void issue(int i, int kt, uint32_t slot) const {
    const uint32_t dst = uni(slot + (wave_of() + NW * i) * 1024);
    if constexpr (!TR) dma16s(voff[i], base + kt * step, dst);
    else dma16s(voff[0], base + kt * step + i * istep, dst);
  }

  // The last stage when it holds only `left` < 64 c: lanes past the end write zeros.
  __device__ __forceinline__ void issue_tail(int kt, int left, char* slot) const {
    const int wave = wave_of(), lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = (wave + NW * i) * RPI + (TR ? lane * 16 / RB : lane / 8);
      const bool in = TR ? r < left : ((lane & 7) ^ swz(r)) * 8 < left;
      if (in) issue(i, kt, (uint32_t)(uintptr_t)slot);
      else *reinterpret_cast<uint4*>(slot + (wave + NW * i) * 1024 + lane * 16) = uint4{0, 0, 0, 0};
    }
  }

  // MFMA fragment of the 32 rows x0.. of k-step ks: lane l gets row l % 32,
  // c = 16 ks + 8 (l / 32) .. + 7
  __device__ __forceinline__ static bf16x8 frag(const char* stage, int x0, int ks) {
    const int lane = threadIdx.x & 63;
    if constexpr (!TR) {
      const int r31 = lane & (TX < 32 ? TX - 1 : 31), r = x0 + r31;
      const int c = (2 * ks + (lane >> 5)) ^ swz(r31);   // x0 is a multiple of 32
      return __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(stage + r * RB + c * 16));
    } else {
      // lane 16 q + i addresses row (i / 4) of its group's four, 8 bytes at
      // column 4 (i % 4), and receives column i of the four rows
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const int i = lane & 15, r = 16 * ks + 8 * (lane >> 5) + (i >> 2);
      const int col = ((lane >> 4) & 1) * 32 + (i & 3) * 8;   // bytes in the 64-byte piece
      const char* p = stage + r * RB + (((x0 / 32) ^ swz(r)) * 64) + col;
      const char* p4 = stage + (r + 4) * RB + (((x0 / 32) ^ swz(r + 4)) * 64) + col;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uint32_t)(uintptr_t)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uint32_t)(uintptr_t)p4);
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    }
  }
};

template <class C, bool TTR, bool FTR>
struct TileG {
  Operand<TTR, C::TM, C::NW> t;
  Operand<FTR, C::TN, C::NW> f;
  f32x16 acc[C::FB][C::TB];

  __device__ __forceinline__ void issue(int i, int kt, uint32_t slot) const {
    if (i < C::NIF) f.issue(i, kt, slot);
    else t.issue(i - C::NIF, kt, slot + C::F_BYTES);
  }

  // One stage of MFMAs; with COPY the copies of stage kt_next spread over the
  // first SP/8 of them. Fragments of k-step ks+1 are read during the MFMAs of
  // k-step ks. Only the first NTB of the wavefront's 32-row blocks are
  // multiplied (the others hold no rows).
  template <bool COPY, int NTB>
  __device__ __forceinline__ void compute(const char* stage, int wf, int wt, int kt_next, uint32_t slot) {
    constexpr int KS = kBK / 16, NMF = C::FB * NTB, NL = C::FB + NTB;
    bf16x8 af[2][C::FB], bf[2][C::TB];
    auto load = [&](int ks, int q) {
      if (q < C::FB) af[ks & 1][q] = f.frag(stage, wf * C::FT + q * 32, ks);
      else bf[ks & 1][q - C::FB] = t.frag(stage + C::F_BYTES, ((q - C::FB) * C::WT + wt) * 32, ks);
    };
#pragma unroll
    for (int q = 0; q < NL; ++q) load(0, q);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
      for (int m = 0; m < NMF; ++m) {
        const int fb = m / NTB, tb = m % NTB;
        acc[fb][tb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[ks & 1][fb], bf[ks & 1][tb], acc[fb][tb], 0, 0, 0);
        if (ks + 1 < KS) {
#pragma unroll
          for (int q = 0; q < NL; ++q)
            if ((q < NMF ? q : NMF - 1) == m) load(ks + 1, q);
        }
        if constexpr (COPY) {
#pragma unroll
          for (int i = 0; i < C::NI; ++i)
            if (C::issue_slot(i, KS * NMF) == ks * NMF + m) issue(i, kt_next, slot);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // Copies of the first stage of `nc` c (with KW > 1, the wavefront's first).
  __device__ __forceinline__ void first(char* lds, int nc, int kw) const {
    const int all = nc / kBK;
    if (kw < all) {
#pragma unroll
      for (int i = 0; i < C::NI; ++i) issue(i, kw, (uint32_t)(uintptr_t)lds);
    } else if (kw == all && nc % kBK) {
      f.issue_tail(kw, nc % kBK, lds);
      t.issue_tail(kw, nc % kBK, lds + C::F_BYTES);
    }
  }

  // All of c, `nc` of them (with KW > 1, the stages kw, kw + KW, ... of them),
  // the first stage's copies already issued.
  template <int NTB>
  __device__ __forceinline__ void mainloop(char* lds, int nc, int wf, int wt, int kw, bool fresh) {
#pragma unroll
    for (int fb = 0; fb < C::FB; ++fb)
#pragma unroll
      for (int tb = 0; tb < C::TB; ++tb) acc[fb][tb] = f32x16{};
    const uint32_t ring = (uint32_t)(uintptr_t)lds;
    const int all = nc / kBK;                                            // whole stages
    const int left = all % C::KW == kw ? nc % kBK : 0;                   // c of this wavefront's short last stage
    const int full = C::KW == 1 ? all : (all - kw + C::KW - 1) / C::KW;  // its whole stages (all >= 0, kw < KW)
    const int nk = full + (left != 0);
    auto at = [&](int s) { return C::KW == 1 ? s : kw + C::KW * s; };
    auto tail = [&](int s) {
      char* slot = lds + (s % C::NS) * C::STAGE;
      f.issue_tail(at(s), left, slot);
      t.issue_tail(at(s), left, slot + C::F_BYTES);
    };
    if constexpr (C::NS > 2) {
      // The other slots may hold the previous tile's staging: every wavefront is
      // past it. Its stores came after the first stage's copies, and are drained
      // so that the counts below see copies only; without stores in between
      // (fresh) all stages are on their way at once.
      if (!fresh) {
        vm_wait<0>();
        if constexpr (C::KW == 1) lds_barrier();
      }
#pragma unroll
      for (int s = 1; s < C::NS - 1; ++s) {
        if (s < full) {
#pragma unroll
          for (int i = 0; i < C::NI; ++i) issue(i, at(s), ring + s * C::STAGE);
        } else if (s < nk) {
          tail(s);
        }
      }
    }
    int slot = 0;
    const int nmain = full - (C::NS - 1);   // stages that copy a later whole stage
    for (int s = 0; s < nmain; ++s) {
      vm_wait<C::NI * (C::NS - 2)>();
      if constexpr (C::KW == 1) lds_barrier();
      const int nslot = slot == 0 ? C::NS - 1 : slot - 1;
      compute<true, NTB>(lds + slot * C::STAGE, wf, wt, at(s + C::NS - 1), ring + nslot * C::STAGE);
      slot = slot + 1 == C::NS ? 0 : slot + 1;
    }
    for (int s = max(nmain, 0); s < nk; ++s) {
      // a short stage's copies are fewer, and zeros written, in some lanes: wait for all
      if (left) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      else vm_wait_ahead<C::NI, C::NS - 2>(nk - 1 - s);
      if constexpr (C::KW == 1) lds_barrier();
      if (left && s + C::NS - 1 == full) tail(full);
      compute<false, NTB>(lds + slot * C::STAGE, wf, wt, 0, 0);
      slot = slot + 1 == C::NS ? 0 : slot + 1;
    }
  }

  // The tile's `rows` rows (at least one): 32-row blocks go to the row
  // wavefronts in turn, so a short tile keeps all of them equally busy with
  // fewer MFMAs.
  __device__ __forceinline__ void multiply(char* lds, int rows, int nc, int wf, int wt, int kw, bool fresh) {
    const int blocks = (min(rows, C::TM) + 32 * C::WT - 1) / (32 * C::WT);
    if constexpr (C::TB >= 2) {
      if (blocks == 1) return mainloop<1>(lds, nc, wf, wt, kw, fresh);
    }
    if constexpr (C::TB >= 3) {
      if (blocks == 2) return mainloop<2>(lds, nc, wf, wt, kw, fresh);
    }
    if constexpr (C::TB >= 4) {
      if (blocks == 3) return mainloop<3>(lds, nc, wf, wt, kw, fresh);
    }
    mainloop<C::TB>(lds, nc, wf, wt, kw, fresh);
  }

  // KW > 1: the wavefronts' sums to LDS, joined in their order and written out.
  __device__ __forceinline__ void store_split(char* lds, void* out, long long ld, int i0, int ni, int j0, int nj, int kw,
                                              bool bf16, bool add) {
    constexpr int ROWB = C::TN * 4, NCH = ROWB / 16;
    const int lane = threadIdx.x & 63;
    char* mine = lds + kw * C::RING;   // this wavefront's ring: it alone used it
#pragma unroll
    for (int fb = 0; fb < C::FB; ++fb)
#pragma unroll
      for (int g4 = 0; g4 < 4; ++g4) {
        const f32x16& v = acc[fb][0];
        *reinterpret_cast<float4*>(mine + stage_off<ROWB>(lane & 31, (fb * 32 + (lane >> 5) * 4 + g4 * 8) * 4)) =
            float4{v[g4 * 4], v[g4 * 4 + 1], v[g4 * 4 + 2], v[g4 * 4 + 3]};
      }
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
      const long long at = (long long)i * ld + col;
      if (bf16) {
        uint2* p = reinterpret_cast<uint2*>(static_cast<__bf16*>(out) + at);
        if (add) {
          const uint2 o = *p;
          s = float4{s.x + bf16_lo(o.x), s.y + bf16_hi(o.x), s.z + bf16_lo(o.y), s.w + bf16_hi(o.y)};
        }
        *p = uint2{pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w)};
      } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        if (add) {
          const float4 o = *p;
          s = float4{s.x + o.x, s.y + o.y, s.z + o.z, s.w + o.w};
        }
        *p = s;
      }
    }
  }

  // Either way out
  __device__ __forceinline__ void write(char* lds, void* out, long long ld, int i0, int ni, int j0, int nj, int wf, int wt,
                                        int kw, bool bf16, bool add) {
    if constexpr (C::KW > 1) {
      store_split(lds, out, ld, i0, ni, j0, nj, kw, bf16, add);
    } else if (bf16) {
      if (add) store<true, true>(lds, out, ld, i0, ni, j0, nj, wf, wt);
      else store<true, false>(lds, out, ld, i0, ni, j0, nj, wf, wt);
    } else {
      if (add) store<false, true>(lds, out, ld, i0, ni, j0, nj, wf, wt);
      else store<false, false>(lds, out, ld, i0, ni, j0, nj, wf, wt);
    }
  }

  // Output rows i0 .. of ni, columns j0 .. of nj: every wavefront stages its 32
  // rows by FT columns in its own LDS and writes whole pieces of 16 bytes, FT
  // columns of a row together. `lds`: staging, behind the first ring slot, which
  // the next tile's copies may be filling. ADD: the sum is added to what is
  // there, in fp32, before the one rounding. (Plain stores: past the caches,
  // weight gradients of 268 MB were 9% faster, but rows that are no whole
  // 128-byte lines took twice as long, 24 x 3344 x 936 bf16 68 against 32 us.)
  template <bool BF16, bool ADD>
  __device__ __forceinline__ void store(char* lds, void* out, long long ld, int i0, int ni, int j0, int nj, int wf,
                                        int wt) {
    constexpr bool PACK = BF16 && !ADD;               // staged as bf16, else as fp32
    constexpr int EB = PACK ? 2 : 4, OB = BF16 ? 2 : 4;   // bytes of a staged and of an output element
    constexpr int ROWB = C::FT * EB, NCH = ROWB / 16, RPP = 64 / NCH;
    const int tid = opaque(threadIdx.x), lane = tid & 63;
    char* mine = lds + C::STAGE + (tid >> 6) * (32 * C::FT * 4);
#pragma unroll
    for (int tb = 0; tb < C::TB; ++tb) {
#pragma unroll
      for (int fb = 0; fb < C::FB; ++fb) {
        f32x16 v = acc[fb][tb];
        asm volatile("" : "+v"(v));
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
          const int col = fb * 32 + (lane >> 5) * 4 + g4 * 8;
          char* p = mine + stage_off<ROWB>(lane & 31, col * EB);
          if constexpr (PACK)
            *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(v[g4 * 4], v[g4 * 4 + 1]), pack_bf16x2(v[g4 * 4 + 2], v[g4 * 4 + 3])};
          else
            *reinterpret_cast<float4*>(p) = float4{v[g4 * 4], v[g4 * 4 + 1], v[g4 * 4 + 2], v[g4 * 4 + 3]};
        }
      }
      // the staging is this wavefront's own: no barrier, only its writes landed
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const int c = lane % NCH, col = j0 + wf * C::FT + c * (16 / EB);
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += RPP) {
        const int r = r0 + lane / NCH, i = i0 + (tb * C::WT + wt) * 32 + r;
        if (i < ni && col < nj) {
          const uint4 v = *reinterpret_cast<const uint4*>(mine + stage_off<ROWB>(r, c * 16));
          char* p = static_cast<char*>(out) + ((long long)i * ld + col) * OB;
          if constexpr (!ADD) {
            *reinterpret_cast<uint4*>(p) = v;
          } else {
            const float4 s = __builtin_bit_cast(float4, v);
            if constexpr (BF16) {
              const uint2 o = *reinterpret_cast<const uint2*>(p);
              *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(bf16_lo(o.x) + s.x, bf16_hi(o.x) + s.y),
                                                   pack_bf16x2(bf16_lo(o.y) + s.z, bf16_hi(o.y) + s.w)};
            } else {
              const float4 o = *reinterpret_cast<const float4*>(p);
              *reinterpret_cast<float4*>(p) = float4{o.x + s.x, o.y + s.y, o.z + s.z, o.w + s.w};
            }
          }
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }
};

// A tile of the call: output rows i0 .. of ni, columns j0 .., nc sums, at `out`.
struct Work {
  int i0, ni, j0, nc;
  char* out;
};

// One workgroup per place on the GPU walks the tiles blockIdx.x, + gridDim.x,
// ...: while a tile is written out the next one's first stage is already on its
// way (a tile of 16 stages spends a fifth of its time on its ends otherwise).
template <class C, int OP>
__global__ void __launch_bounds__(C::THREADS, (C::THREADS / 256) * C::OCC) moe_gemm_bf16(const GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  constexpr bool WG = OP == MOE_GROUPED_WGRAD, FWD = OP == MOE_GROUPED_FORWARD;
  const int wave = uni((int)(threadIdx.x >> 6)), kw = C::KW == 1 ? 0 : wave;
  const int wf = C::KW == 1 ? wave % C::WF : 0, wt = C::KW == 1 ? wave / C::WF : 0;
  char* const ring = lds + kw * C::RING;
  TileG<C, WG, !FWD> g;
  const __bf16* x = static_cast<const __bf16*>(a.x);
  const __bf16* w = static_cast<const __bf16*>(a.w);
  const __bf16* y = static_cast<const __bf16*>(a.y);
  const int nj = FWD ? a.n : a.k;                    // output columns
  const int tj = (nj + C::TN - 1) / C::TN;           // tiles along them
  const int ti = WG ? (a.n + C::TM - 1) / C::TM : 0; // wgrad: tiles along an expert's rows of W
  const long long ldt = FWD ? a.ld_x : a.ld_y, ldo = WG ? a.ld_w : FWD ? a.ld_y : a.ld_x;
  const int oe = a.out_bf16 ? 2 : 4;
  const GroupScan<C::TM> scan(a.row_offset, a.L, a.rows);
  const int tiles = WG ? a.L * ti * tj : scan.total * tj, total = tiles * a.splits;

  // tile of workgroup slot b: what it is, and the copies of its first stage
  auto start = [&](int b, Work& wk) {
    int tile = xcd_tile(b, total);
    if (tile >= total) return false;
    int s = 0, c0 = 0;
    if (a.splits > 1) {
      s = tile / tiles;
      tile -= s * tiles;
    }
    if constexpr (WG) {
      const int e = tile / (ti * tj);
      int i, j;
      tile_at(tile - e * ti * tj, ti, tj, i, j);
      const int r0 = uni(clamped_offset(a.row_offset, a.L, a.rows, e));
      const int Me = uni(max(clamped_offset(a.row_offset, a.L, a.rows, e + 1) - r0, 0));
      const int nc = split_range<kBK>(Me, a.splits, s, c0);
      wk = Work{i * C::TM, a.n, j * C::TN, nc, static_cast<char*>(a.w) + ((long long)e * a.es_w + s * a.part) * oe};
      g.t.setup(y + (long long)(r0 + c0) * a.ld_y, a.ld_y, wk.i0, a.n);
      g.f.setup(x + (long long)(r0 + c0) * a.ld_x, a.ld_x, wk.j0, a.k);
    } else {
      int p, j;
      tile_at(tile, scan.total, tj, p, j);
      const Group gr = scan.find(p);
      const int nc = split_range<kBK>(FWD ? a.k : a.n, a.splits, s, c0);
      wk = Work{gr.m * C::TM, gr.Me, j * C::TN, nc,
                static_cast<char*>(FWD ? a.y : a.x) + ((long long)gr.r0 * ldo + s * a.part) * oe};
      g.t.setup((FWD ? x : y) + (long long)gr.r0 * ldt + c0, ldt, wk.i0, wk.ni);
      g.f.setup(w + (long long)gr.e * a.es_w + (FWD ? c0 : (long long)c0 * a.ld_w), a.ld_w, wk.j0, nj);
    }
    g.first(ring, wk.nc, kw);
    return true;
  };

  Work cur, next;
  int b = blockIdx.x;
  bool more = start(b, cur), fresh = true;
  while (more) {
    g.multiply(ring, cur.ni - cur.i0, cur.nc, wf, wt, kw, fresh);
    fresh = C::KW > 1;   // split wavefronts store before they copy
    b += gridDim.x;
    const bool write = !WG || cur.nc > 0 || !a.accumulate;
    if constexpr (C::KW == 1) {
      lds_barrier();   // every wavefront is done with the ring
      more = start(b, next);
      if (write) g.write(lds, cur.out, ldo, cur.i0, cur.ni, cur.j0, nj, wf, wt, kw, a.out_bf16, a.accumulate);
    } else {
      if (write) g.write(lds, cur.out, ldo, cur.i0, cur.ni, cur.j0, nj, wf, wt, kw, a.out_bf16, a.accumulate);
      __syncthreads();   // the joined sums are read
      more = start(b, next);
    }
    // the staging's LDS writes and reads, and a short first stage's zeros, are
    // this wavefront's own and done; the next loop's barrier publishes them
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    cur = next;
  }
}

//                   rows cols  wavefronts ring spread workgroups per CU
using Large = CfgG<256, 256, 2, 4, 2, 2, 1>;
using Wide = CfgG<192, 256, 2, 4, 2, 2, 1>;
using Medium = CfgG<128, 256, 2, 4, 3, 4, 1>;
using Square = CfgG<128, 128, 2, 2, 2, 4, 2>;
// one workgroup per CU with four stages: 4 to 19% faster than Square where no
// compute unit gets a second tile (1024 x 4096 x 4096: 36 against 45 us), never
// the fastest where one does
using Deep = CfgG<128, 128, 2, 4, 4, 4, 1>;
using Small = CfgG<64, 128, 1, 4, 3, 4, 2>;
using Split = CfgG<32, 32, 1, 1, 2, 4, 1, 8>;
using Split64 = CfgG<32, 64, 1, 1, 3, 4, 1, 4>;
using Few = CfgG<16, 32, 1, 1, 3, 4, 1, 8>;   // few rows: fewer bytes a stage, more stages on their way

template <class C>
constexpr GemmTile timed(double a, double c, double b, double o, bool once = false) {
  return GemmTile{C::TM, C::TN, C::OCC, C::KW, a, c, b, o, once};
}

template <class C, int OP>
hipError_t launch(const GemmArgs& a, hipStream_t s) {
  const long long nj = ((OP == MOE_GROUPED_FORWARD ? a.n : a.k) + C::TN - 1) / C::TN;
  const long long mi = OP == MOE_GROUPED_WGRAD ? (long long)a.L * ((a.n + C::TM - 1) / C::TM)
                                               : ((long long)a.rows + (long long)a.L * (C::TM - 1)) / C::TM;
  const long long tiles = nj * mi * a.splits;
  if (tiles >= INT_MAX / 2) return launch_gemm_any(a, false, s);   // the kernel counts tiles in int
  // A workgroup for each place on the GPU; a multiple of 8 keeps one on its XCD.
  // Past a tile for every compute unit all places get one, since the tile order
  // is dealt in runs: with a workgroup for each of 288 to 320 tiles, places for
  // the last ones stayed empty (2048 x 4096 x 2304 in 128 x 128: 84 us, now 52).
  const long long grid = tiles > kCus ? kCus * C::OCC : (tiles + 7) / 8 * 8;
  moe_gemm_bf16<C, OP><<<(unsigned)grid, C::THREADS, 0, s>>>(a);
  return hipGetLastError();
}

template <int OP>
hipError_t launch_tile(int id, const GemmArgs& a, hipStream_t s) {
  switch (id) {
    case 1: return launch<Large, OP>(a, s);
    case 3: return launch<Medium, OP>(a, s);
    case 4: return launch<Square, OP>(a, s);
    case 5: return launch<Small, OP>(a, s);
  }
  // not wgrad: its operands' LDS rows are a tile's columns, 1024 bytes must
  // hold whole ones, and its tiles are many enough without splitting the sum
  if constexpr (OP != MOE_GROUPED_WGRAD) {
    switch (id) {
      case 2: return launch<Wide, OP>(a, s);
      case 6: return launch<Split, OP>(a, s);
      case 7: return launch<Split64, OP>(a, s);
      case 8: return launch<Deep, OP>(a, s);
      case 9: return launch<Few, OP>(a, s);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace

// forward; dgrad, whose narrow tiles read half lines of the weights; wgrad (both
// operands through transposing reads)
const GemmTile kBf16GemmTileTable[] = {
    timed<Large>(0.84, 1.56, 1.56, 4),  timed<Wide>(0.73, 1.27, 1.27, 4),  timed<Medium>(0.48, 0.90, 0.90, 5),
    timed<Square>(0.47, 0.79, 0.54, 2), timed<Small>(0.22, 0.37, 0.32, 4), timed<Split>(0.78, 0.96, 0.96, 1),
    timed<Split64>(0.52, 0.64, 0.64, 2), timed<Deep>(0.28, 0.48, 0.48, 5, true), timed<Few>(0.64, 0.64, 0.64, 1)};
const GemmTile kDgradTiles[] = {
    timed<Large>(0.78, 1.56, 1.56, 5),  timed<Wide>(0.73, 1.27, 1.27, 5),  timed<Medium>(0.48, 0.90, 0.90, 6),
    timed<Square>(0.54, 0.79, 0.54, 2), timed<Small>(0.25, 0.37, 0.32, 4), timed<Split>(0.78, 1.18, 1.18, 1),
    timed<Split64>(0.56, 0.73, 0.73, 2), timed<Deep>(0.30, 0.52, 0.52, 4, true), timed<Few>(0.73, 1.03, 1.03, 1)};
const GemmTile kWgradTiles[] = {
    timed<Large>(1.10, 1.79, 1.79, 6),  GemmTile{}, timed<Medium>(0.60, 0.96, 0.96, 4),
    timed<Square>(0.47, 0.70, 0.47, 4), timed<Small>(0.32, 0.32, 0.32, 3), GemmTile{}, GemmTile{}, GemmTile{}, GemmTile{}};

hipError_t launch_gemm_bf16(int id, const GemmArgs& a, hipStream_t s) {
  switch (a.op) {
    case MOE_GROUPED_FORWARD: return launch_tile<MOE_GROUPED_FORWARD>(id, a, s);
    case MOE_GROUPED_DGRAD: return launch_tile<MOE_GROUPED_DGRAD>(id, a, s);
    default: return launch_tile<MOE_GROUPED_WGRAD>(id, a, s);
  }
}

}  // namespace moe
