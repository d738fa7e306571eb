// Block-scaled e4m3 matrix products, dense or grouped by expert, for 16-byte
// aligned operands:
//
//   y(r, n) = sum over 128-wide K blocks b of xs(r, b) ws(n/128, b) P_b(r, n),
//   P_b(r, n) = sum over k in b of x(r, k) w(n, k)
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 (unit scales) is one P_b of a 16 x 16
// block: the fp32 scales are no powers of two and cannot ride in the MFMA, so
// the VALU adds each P_b into the accumulator times its scales, two MFMAs
// behind the matrix core (four FMAs a lane under a 32-cycle MFMA). Weights are
// the A operand and rows the B operand: a lane holds one row and runs of four
// consecutive n, its row scale is one register and its weight scale is uniform.
//
// The e4m3 MFMAs (this one and the unscaled 16x16x32 alike, measured) add eight
// consecutive products after dropping each one's bits below 2^-13 of the
// largest's power of two: about 1.5e-5 of a result, against the 2^-4 half step
// of the operands. Products through bf16 MFMAs would keep those bits at half
// the rate and with a conversion of every operand, and were not taken.
//
// A stage is one K block (128 bytes a row): an NS-deep LDS ring filled by
// direct-to-LDS copies between the MFMAs of an earlier stage; the stage's row
// scales come along as four-byte copies, and the weight scales by a wavefront
// that has no rows left to fetch scales for (a load to registers would wait for
// every copy and store in flight). A ragged last block is zeros in LDS.

#include "internal.hpp"
#include "ops_common.hpp"

namespace moe {
namespace {

// 16 (or 4) bytes a lane from base + voff (bytes) to LDS m0 + 16 (4) * lane;
// s_nop: m0's wait state (see dma16 in ffn_common.hpp)
__device__ __forceinline__ void dma16s(uint32_t voff, const char* base, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(m0) : "memory", "m0");
}
__device__ __forceinline__ void dma4s(uint32_t voff, const char* base, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "s"(m0) : "memory", "m0");
}

// KW > 1: KW wavefronts split K (see the bf16 kernel): a ring each, sums joined in LDS.
template <int TM_, int TN_, int WT_, int WF_, int NS_, int SP_, int OCC_, int KW_ = 1>
struct CfgQ {
  static constexpr int TM = TM_, TN = TN_, WT = WT_, WF = WF_, NS = NS_, SP = SP_, OCC = OCC_;
  static constexpr int KW = KW_, NW = WT * WF, THREADS = 64 * NW * KW;
  static constexpr int TT = TM / WT, FT = TN / WF;
  static constexpr int TB = TT / 16, FB = FT / 16, NB = TB * FB;   // 16 x 16 blocks of a wavefront
  static constexpr int TP = TB > 1 ? TB / 2 : 1;                   // 32-row blocks
  static constexpr int NIT = TM * 128 / 1024 / NW, NIF = TN * 128 / 1024 / NW;
  static constexpr int NS_COPIES = KW > 1 ? 2 : 1;       // scales: rows', and weights' where no wavefront is left for them
  static constexpr int NI = NIT + NIF + NS_COPIES;
  static constexpr int F_BYTES = TN * 128, T_BYTES = TM * 128, S_BYTES = (NW + NS_COPIES - 1) * 256;
  static constexpr int STAGE = F_BYTES + T_BYTES + S_BYTES;
  static constexpr int EPI = NW * 16 * FT * 4;
  static constexpr int RING = NS * STAGE;
  static constexpr int LDS = KW * RING;
  static_assert(RING - STAGE >= EPI || KW > 1, "the epilogue stages behind the next tile's first stage");
  static_assert(KW == 1 || (NW == 1 && TM <= 32), "split wavefronts hold the whole tile each");
  // copies of a stage when only ntp 32-row blocks a wavefront hold rows, the
  // scales' last
  static constexpr int copies(int ntp) { return NIF + NIT * ntp / TP + NS_COPIES; }
  static constexpr int issue_slot(int i, int nb, int ni) { return i * nb * SP / (ni * 8); }
  static_assert(NIT % TP == 0, "copies of a row block");
  static constexpr int NP = NB < 4 ? NB : 4;             // products in flight
  static_assert(16 * FT * 2 % 1024 == 0 || KW > 1, "a 16-row piece of the epilogue is whole stores");
  static_assert(FT <= 128 && 128 % FT == 0, "a wavefront's columns lie in one block of weight scales");
  static_assert(NB % NP == 0 && TB == 2 * TP - (TB == 1) && FB >= 2 && (NB > 2 || FB == 2), "blocks of a wavefront");
  static_assert(TM < 64 * NW || KW > 1, "row-scale copies cover the tile, a wavefront is left for the weight scales");
  static_assert((TM * 128) % (1024 * NW) == 0 && (TN * 128) % (1024 * NW) == 0, "copies split evenly");
  static_assert(NS >= 2 && NI * (NS - 1) <= 63, "vmcnt range");
  static_assert(LDS * OCC <= 160 * 1024, "LDS");
};

// Physical 16-byte chunk of logical chunk c in row r of a stage, and back: the
// fragment reads take rows r16 at chunks 2g and 2g+1 (g = lane / 16), and this
// bijection spreads both over all banks (measured without conflicts).
__device__ __forceinline__ int chunk_at(int r, int c) { return c ^ ((r >> 1) & 7) ^ ((c & 2) << 1); }
__device__ __forceinline__ int chunk_in(int r, int p) {
  const int q = p ^ ((r >> 1) & 7);
  return q ^ ((q & 2) << 1);
}

template <class C>
struct TileQ {
  const char *fbase, *tbase, *sbase, *wbase;
  uint32_t fv[C::NIF], tv[C::NIT], sv;
  f32x4 acc[C::FB][C::TB];
  f32x4 part[C::NP];
  float s_tail[2];

  __device__ __forceinline__ static int wave_of() { return C::NW == 1 ? 0 : uni((int)(threadIdx.x >> 6)); }

  template <int NI>
  __device__ __forceinline__ static void offsets(uint32_t (&v)[NI], long long ld, int last) {
    const int wave = wave_of(), lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = (wave + C::NW * i) * 8 + lane / 8;
      v[i] = (uint32_t)min(r, last) * (uint32_t)ld + chunk_in(r, lane & 7) * 16;
    }
  }

  __device__ __forceinline__ void issue(int i, int kt, uint32_t slot) const {
    const uint32_t wave = wave_of();
    slot = uni(slot);
    if (i < C::NIF) dma16s(fv[i], fbase + kt * 128ll, slot + (wave + C::NW * i) * 1024);
    else if (i < C::NIF + C::NIT) dma16s(tv[i - C::NIF], tbase + kt * 128ll, slot + C::F_BYTES + (wave + C::NW * (i - C::NIF)) * 1024);
    else if (i == C::NIF + C::NIT) dma4s(sv, sbase + kt * 4ll, slot + C::F_BYTES + C::T_BYTES + wave * 256);
    else dma4s(0, wbase + kt * 4ll, slot + C::F_BYTES + C::T_BYTES + 256);
  }

  // the last block when it holds only `left` < 128 k: lanes past it write zeros
  __device__ __forceinline__ void issue_tail(int kt, int left, char* slot) const {
    const int wave = wave_of(), lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < C::NIF + C::NIT; ++i) {
      const int j = i < C::NIF ? i : i - C::NIF;
      const int r = (wave + C::NW * j) * 8 + lane / 8;
      const bool in = chunk_in(r, lane & 7) * 16 < left;
      if (in) issue(i, kt, (uint32_t)(uintptr_t)slot);
      else *reinterpret_cast<uint4*>(slot + (i < C::NIF ? 0 : C::F_BYTES) + (wave + C::NW * j) * 1024 + lane * 16) = uint4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = C::NIF + C::NIT; i < C::NI; ++i) issue(i, kt, (uint32_t)(uintptr_t)slot);
  }

  __device__ __forceinline__ static i32x8 frag(const char* stage, int r, int c) {
    const char* row = stage + r * 128;
    const uint4 lo = *reinterpret_cast<const uint4*>(row + (chunk_at(r, c) << 4));
    const uint4 hi = *reinterpret_cast<const uint4*>(row + (chunk_at(r, c + 1) << 4));
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  }

  // One K block. The products of the stage's last two blocks are added during
  // the first two MFMAs of the next one. Only the first NTP of the wavefront's
  // 32-row blocks are multiplied.
  template <bool COPY, int NTP>
  __device__ __forceinline__ void compute(const char* stage, int wf, int wt, int kt_next, uint32_t slot) {
    constexpr int TB = C::TB == 1 ? 1 : 2 * NTP, NB = C::FB * TB, NI = C::copies(NTP);
    // row of 16-row block j: 32-row blocks go to the row wavefronts in turn
    auto row = [&](int j) { return ((j >> 1) * C::WT + wt) * 32 + (j & 1) * 16; };
    const int lane = threadIdx.x & 63, r16 = lane & 15, c0 = 2 * (lane >> 4);
    const char* ts = stage + C::F_BYTES;
    const float* sx = reinterpret_cast<const float*>(ts + C::T_BYTES) + r16;
    // behind the row scales, or (KW > 1) behind their 256 bytes
    const float sw = *(reinterpret_cast<const float*>(ts + C::T_BYTES) + (C::KW > 1 ? 64 : C::TM + wf * C::FT / 128));
    i32x8 af[C::FB], bf[2];
    float st[2];
    bf[0] = frag(ts, row(0) + r16, c0);
    af[0] = frag(stage, wf * C::FT + r16, c0);
    st[0] = sx[row(0)] * sw;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int j = b / C::FB, i = b % C::FB;
      if (b + 1 < C::FB) af[b + 1] = frag(stage, wf * C::FT + (b + 1) * 16 + r16, c0);
      if (i == 0 && j + 1 < TB) bf[(j + 1) & 1] = frag(ts, row(j + 1) + r16, c0);
      if constexpr (NB == 2) {   // before its place is taken
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[b][0][v] += part[b][v] * s_tail[b];
      }
      part[b % C::NP] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af[i], bf[j & 1], f32x4{}, 0, 0, 0, 127, 0, 127);
      const int q = b - 2;
      if constexpr (NB == 2) {
      } else if (q >= 0) {
        const float s = st[(q / C::FB) & 1];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[q % C::FB][q / C::FB][v] += part[q % C::NP][v] * s;
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[C::FB + q][TB - 1][v] += part[(q + C::NP) % C::NP][v] * s_tail[q + 2];
      }
      // the next rows' scale once the last use of the one it replaces is past
      if (i == (C::FB > 2 ? 2 : 1) && j + 1 < TB) st[(j + 1) & 1] = sx[row(j + 1)] * sw;
      if constexpr (COPY) {
#pragma unroll
        for (int k = 0; k < NI; ++k)
          if (C::issue_slot(k, NB, NI) == b) issue(k + C::NS_COPIES >= NI ? C::NI - NI + k : k, kt_next, slot);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    s_tail[0] = s_tail[1] = st[(TB - 1) & 1];
  }

  // Copies of the first block of K (with KW > 1, the wavefront's first)
  __device__ __forceinline__ void first(char* lds, int K, int kw) const {
    if (kw < K / 128) {
#pragma unroll
      for (int i = 0; i < C::NI; ++i) issue(i, kw, (uint32_t)(uintptr_t)lds);
    } else if (kw == K / 128 && K % 128) {
      issue_tail(kw, K % 128, lds);
    }
  }

  // All of K (with KW > 1, blocks kw, kw + KW, ...), the first stage's copies
  // already issued
  template <int NTP>
  __device__ __forceinline__ void mainloop(char* lds, int K, int wf, int wt, int kw, int stores, bool fresh) {
    constexpr int NI = C::copies(NTP);
#pragma unroll
    for (int i = 0; i < C::FB; ++i)
#pragma unroll
      for (int j = 0; j < C::TB; ++j) acc[i][j] = f32x4{};
    // the first stage adds the products before it: nothing, exactly
#pragma unroll
    for (int i = 0; i < C::NP; ++i) part[i] = f32x4{};
    s_tail[0] = s_tail[1] = 0.f;
    const uint32_t ring = (uint32_t)(uintptr_t)lds;
    const int all = K / 128;
    const int left = all % C::KW == kw ? K % 128 : 0;
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
          for (int i = 0; i < NI; ++i) issue(i + C::NS_COPIES >= NI ? C::NI - NI + i : i, at(s), ring + s * C::STAGE);
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
    if (nk > 0) {
      constexpr int TB = C::TB == 1 ? 1 : 2 * NTP, NB = C::FB * TB;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        acc[C::FB - 2][TB - 1][v] += part[(NB - 2) % C::NP][v] * s_tail[0];
        acc[C::FB - 1][TB - 1][v] += part[(NB - 1) % C::NP][v] * s_tail[1];
      }
    }
  }

  // The tile's `rows` rows (at least one)
  __device__ __forceinline__ void multiply(char* lds, int rows, int K, int wf, int wt, int kw, int stores,
                                           bool fresh) {
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

  // KW > 1: the wavefronts' sums to LDS, joined in their order and written out.
  __device__ __forceinline__ void store_split(char* lds, void* out, long long ld, int i0, int ni, int j0, int nj, int kw,
                                              bool bf16) {
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
      if (bf16) *reinterpret_cast<uint2*>(static_cast<__bf16*>(out) + p) = uint2{pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w)};
      else *reinterpret_cast<float4*>(static_cast<float*>(out) + p) = s;
    }
  }

  // Rows i0 .. of ni, columns j0 .. of nj (see the bf16 kernel's store), 16 rows at a time
  template <bool BF16>
  static constexpr int STORES = C::TB * 16 * (C::FT * (BF16 ? 2 : 4) / 16) / 64;

  template <bool BF16, bool WHOLE>
  __device__ __forceinline__ void store(char* lds, void* out, long long ld, int i0, int ni, int j0, int nj, int wf, int wt) {
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
        if (WHOLE || (r < 16 && i < ni && col < nj))
          *reinterpret_cast<uint4*>(static_cast<char*>(out) + ((long long)i * ld + col) * EB) =
              *reinterpret_cast<const uint4*>(mine + stage_off<ROWB>(r, c * 16));
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }

  // the stores that the wavefront issued, or 0 if it does not know
  __device__ __forceinline__ int write(char* lds, void* out, long long ld, int i0, int ni, int j0, int nj, int wf, int wt,
                                       bool bf16) {
    if (i0 + C::TM <= ni && j0 + C::TN <= nj) {
      if (bf16) return store<true, true>(lds, out, ld, i0, ni, j0, nj, wf, wt), STORES<true>;
      return store<false, true>(lds, out, ld, i0, ni, j0, nj, wf, wt), STORES<false>;
    }
    if (bf16) store<true, false>(lds, out, ld, i0, ni, j0, nj, wf, wt);
    else store<false, false>(lds, out, ld, i0, ni, j0, nj, wf, wt);
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
__global__ void __launch_bounds__(C::THREADS, (C::THREADS / 256) * C::OCC) moe_gemm_fp8(const GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  const int wave = uni((int)(threadIdx.x >> 6)), kw = C::KW == 1 ? 0 : wave, lane = threadIdx.x & 63;
  const int wf = C::KW == 1 ? wave % C::WF : 0, wt = C::KW == 1 ? wave / C::WF : 0;
  char* const ring = lds + kw * C::RING;
  const int tj = (a.n + C::TN - 1) / C::TN, kb = (a.k + 127) / 128, nb = (a.n + 127) / 128;
  const int oe = a.out_bf16 ? 2 : 4;
  const bool grouped = a.row_offset != nullptr;
  const GroupScan<C::TM> scan(a.row_offset, grouped ? a.L : 0, a.rows);
  const int ti = grouped ? scan.total : (a.rows + C::TM - 1) / C::TM;
  const int tiles = ti * tj, total = tiles * a.splits;
  TileQ<C> g;

  auto start = [&](int b, Work& wk) {
    int tile = xcd_tile(b, total);
    if (tile >= total) return false;
    int s = 0, c0 = 0;
    if (a.splits > 1) {
      s = tile / tiles;
      tile -= s * tiles;
    }
    const int nc = split_range<128>(a.k, a.splits, s, c0);
    int p, j;
    tile_at(tile, ti, tj, p, j);
    const Group gr = grouped ? scan.find(p) : Group{0, p, 0, a.rows, true};
    const int i0 = gr.m * C::TM, j0 = j * C::TN;
    g.fbase = static_cast<const char*>(a.w) + (long long)gr.e * a.es_w + (long long)j0 * a.ld_w + c0;
    g.tbase = static_cast<const char*>(a.x) + (long long)(gr.r0 + i0) * a.ld_x + c0;
    g.offsets(g.fv, a.ld_w, a.n - 1 - j0);
    g.offsets(g.tv, a.ld_x, gr.Me - 1 - i0);
    // scales: rows wave * 64 + lane of the tile, behind them the tile's blocks of weights
    const long long wblock = (long long)gr.e * nb + j0 / 128;
    const int srow = g.wave_of() * 64 + lane;
    if (C::KW > 1 || g.wave_of() * 64 < C::TM) {
      g.sbase = reinterpret_cast<const char*>(a.xs + (long long)(gr.r0 + i0) * a.ld_xs + c0 / 128);
      g.sv = (uint32_t)min(srow % C::TM, gr.Me - 1 - i0) * (uint32_t)(a.ld_xs * 4);
    } else {
      g.sbase = reinterpret_cast<const char*>(a.ws + wblock * kb + c0 / 128);
      g.sv = (uint32_t)min(srow - C::TM, min(1, nb - 1 - j0 / 128)) * (uint32_t)(kb * 4);
    }
    g.wbase = reinterpret_cast<const char*>(a.ws + wblock * kb + c0 / 128);
    wk = Work{i0, gr.Me, j0, nc,
              static_cast<char*>(a.y) + ((long long)gr.r0 * a.ld_y + s * a.part) * oe};
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
      stores = g.write(lds, cur.out, a.ld_y, cur.i0, cur.ni, cur.j0, a.n, wf, wt, a.out_bf16);
    } else {
      g.store_split(lds, cur.out, a.ld_y, cur.i0, cur.ni, cur.j0, a.n, kw, a.out_bf16);
      __syncthreads();   // the joined sums are read
      more = start(b, next);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    cur = next;
  }
}

//                   rows cols  wavefronts ring spread workgroups per CU
using Large = CfgQ<256, 256, 2, 4, 2, 4, 1>;
using Wide = CfgQ<192, 256, 2, 4, 2, 4, 1>;
using Medium = CfgQ<128, 256, 2, 4, 3, 4, 1>;
using Square = CfgQ<128, 128, 2, 2, 2, 4, 2>;
using Deep = CfgQ<128, 128, 2, 4, 4, 4, 1>;   // for calls that give no compute unit a second tile
using Small = CfgQ<64, 128, 1, 4, 3, 4, 2>;
using Split = CfgQ<32, 32, 1, 1, 2, 4, 1, 8>;
using Split64 = CfgQ<32, 64, 1, 1, 3, 4, 1, 4>;
using Few = CfgQ<16, 32, 1, 1, 3, 4, 1, 8>;   // few rows: fewer bytes a stage, more stages on their way

template <class C>
constexpr GemmTile timed(double a, double c, double b, double o, bool once = false) {
  return GemmTile{C::TM, C::TN, C::OCC, C::KW, a, c, b, o, once};
}

template <class C>
hipError_t launch(const GemmArgs& a, hipStream_t s) {
  const long long tiles = gemm_tiles(a, C::TM, C::TN);
  if (tiles >= kMostTiles) return launch_gemm_any(a, true, s);   // only whole sums (ops_api.cpp)
  const long long grid = tiles > kCus ? kCus * C::OCC : (tiles + 7) / 8 * 8;
  moe_gemm_fp8<C><<<(unsigned)grid, C::THREADS, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

const GemmTile kFp8GemmTileTable[] = {
    timed<Large>(0.73, 1.67, 1.67, 6),  timed<Wide>(0.68, 1.36, 1.36, 5),  timed<Medium>(0.60, 0.96, 0.96, 5),
    timed<Square>(0.37, 0.79, 0.54, 4), timed<Small>(0.28, 0.42, 0.32, 4), timed<Split>(0.68, 0.68, 0.68, 2),
    timed<Split64>(0.60, 0.68, 0.68, 2), timed<Deep>(0.37, 0.56, 0.56, 5, true), timed<Few>(0.50, 0.64, 0.64, 2)};

hipError_t launch_gemm_fp8(int id, const GemmArgs& a, hipStream_t s) {
  switch (id) {
    case 1: return launch<Large>(a, s);
    case 2: return launch<Wide>(a, s);
    case 3: return launch<Medium>(a, s);
    case 4: return launch<Square>(a, s);
    case 5: return launch<Small>(a, s);
    case 6: return launch<Split>(a, s);
    case 7: return launch<Split64>(a, s);
    case 8: return launch<Deep>(a, s);
    case 9: return launch<Few>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
