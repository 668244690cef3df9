// The large tile of the ragged grouped products: BN output columns x BM output rows per workgroup,
// operands brought from memory straight into two rings of LDS stages.
//
// A stage is 128 bytes of the sum index of one operand (the image of moe_product.h). Whole stages
// are copied by the DMA form of the global load (16 bytes per lane, 1 KB of consecutive LDS per
// wave and instruction; the image's swizzle is applied by choosing which chunk a lane fetches),
// NSN - 1 (n operand) and NSM - 1 (m operand) stages ahead of the MFMAs. In a last, partial stage (a
// sum length that is no multiple of a stage, and every expert's rows in a weight gradient) the
// lanes whose chunk lies behind the end fetch 16 zero bytes instead. Rows and columns behind the
// tile's edge are fetched from its last row or chunk and never stored.
//
// Order. Each of a stage's two MFMA steps multiplies fragments that were read during the step
// before it; between its MFMAs go the LDS reads of the next step and half of the loads of the
// stages ahead, one by one: a wave issues in order, and a run of loads stalls it (and its MFMAs)
// at the rate the memory path takes them, 16 clocks per KB.
//
// Waits. The compiler does not order the direct LDS writes against LDS reads. Loads return in issue
// order, so at point j (before the last MFMA step of stage j - 1) a count says that this wave's
// parts of stage j are in LDS; the barrier after it says so for all waves, and that every wave has
// read its fragments of stage j - 1, whose ring slots the loads issued next overwrite.
//
// Measured (one MI355X, random normals). 8192^3 bf16: forward 1250, input gradient 1460, weight
// gradient 1350 TFLOP/s, int8 2305 TOP/s; the vendor library on the same shapes 1210 / 1520 / 1080
// and 2100. What bounds it is power: the input gradient keeps the matrix units busy 78% of its
// cycles at 1.69 GHz, the library's kernel 92% at 1.56 GHz. That is why the 16 x 16 MFMA is taken:
// it sums twice the k of the 32 x 32 form into each accumulator it touches (input gradient 1280 with
// 32 x 32). Four waves with 128 x 128 each read a third less LDS than eight with 128 x 64 (1256
// against 1206, before the loads were spread), and loads spread between the MFMAs took it from
// 62% to 78% busy.
#pragma once

#include "moe_gemm_big.h"
#include "moe_product.h"

namespace moe {
namespace {

// 16-byte direct load of one lane to LDS from a uniform base and a 32-bit lane offset; the wave's
// lanes fill 1 KB from LDS byte address `l`. Written as assembly because the compiler would put a
// wait for every direct load in flight before each transposing LDS read (it cannot tell their
// places apart). Nothing but LDS is written, and the compiler's own counted waits only get
// stricter by loads it does not count. (One idle state between the write of M0 and its use. M0 is
// no allocatable register: the compiler sets it where it needs it itself.)
__device__ __forceinline__ void dma16_at(const uint8_t* base, uint32_t off, uint32_t l) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(l), "v"(off), "s"(base)
               : "memory");
#else
  (void)base, (void)off, (void)l;
#endif
}

// the same from a 64-bit lane address
__device__ __forceinline__ void dma16_from(const uint8_t* g, uint32_t l) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(l), "v"(g)
               : "memory");
#else
  (void)g, (void)l;
#endif
}

// what lanes behind the end of a sum fetch
__device__ __attribute__((aligned(16))) const uint8_t kZeroChunk[16] = {};

// byte address of a place in LDS
__device__ __forceinline__ uint32_t lds_address(const uint8_t* l) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) const uint8_t lds_u8_t;
  return (uint32_t)(uintptr_t)(lds_u8_t*)l;
#else
  (void)l;
  return 0;
#endif
}

// c is in accumulator registers here. The tile's 256 sums per lane are all of them; pinned at every
// step they stay there, while left to itself the compiler moves some through vector registers and
// scratch around every MFMA. (The MFMAs themselves stay the compiler's: it keeps the waits that
// reading a result too early would need.)
template <class Acc>
__device__ __forceinline__ void acc_pin(Acc& c) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+a"(c));
#endif
}

// ------------------------------------------------------------------------------------------------
// M tiles without LDS (the rings may fill it): every wave holds the first tile of up to 16 experts
// per lane and finds a tile's expert by ballots.
// ------------------------------------------------------------------------------------------------
struct WaveTiles {
  int epl;    // experts per lane
  int first;  // tiles before expert lane * epl
  int total;
};

__device__ __forceinline__ WaveTiles wave_tiles(const ProductArgs& p, int bm) {
  WaveTiles x;
  const int lane = threadIdx.x & 63;
  x.epl = (p.E + 63) / 64;
  int cnt = 0;
  for (int q = 0; q < x.epl; ++q) {
    const int e = lane * x.epl + q;
    if (e < p.E) {
      int lo, hi;
      expert_rows(p, e, lo, hi);
      cnt += (hi - lo + bm - 1) / bm;
    }
  }
  int inc = cnt;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  x.first = inc - cnt;
  x.total = __builtin_amdgcn_readlane(inc, 63);
  return x;
}

struct TileAt {
  int e, row0, row_end, n0;
};

// expert and rows of M tile ti (< total), uniform: the last lane whose experts start at or before
// ti holds it, and of that lane's experts (one per lane now) again the last
__device__ __forceinline__ void wave_lookup(const ProductArgs& p, const WaveTiles& x, int ti,
                                            int bm, TileAt& at) {
  const int lane = threadIdx.x & 63;
  const int sel = 63 - __builtin_clzll(__ballot(x.first <= ti));
  const int e = sel * x.epl + lane;
  const bool mine = lane < x.epl && e < p.E;
  int lo = 0, hi = 0;
  if (mine) expert_rows(p, e, lo, hi);
  const int cnt = (hi - lo + bm - 1) / bm;
  int inc = cnt;
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  const int start = __builtin_amdgcn_readlane(x.first, sel) + inc - cnt;
  const int pick = 63 - __builtin_clzll(__ballot(mine && start <= ti));
  at.e = sel * x.epl + pick;
  at.row0 = __builtin_amdgcn_readlane(lo, pick) + (ti - __builtin_amdgcn_readlane(start, pick)) * bm;
  at.row_end = __builtin_amdgcn_readlane(hi, pick);
}

template <int EL, int NK, int MK, int BN, int BM, int WN, int WM, int NSN, int NSM>
struct ProductBig {
  static constexpr int kWaves = WN * WM;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int TN = BN / WN, TM = BM / WM;  // a wave's tile
  static constexpr int NI = TN / 16, NJ = TM / 16;
  static constexpr int NQ = BN * 8 / kThreads;      // 16-byte chunks per thread and stage
  static constexpr int MQ = BM * 8 / kThreads;
  static constexpr int EB = ProductTypes<EL>::kBytes;
  static constexpr int BK = 128 / EB;
  static constexpr int kNStage = BN * 128, kMStage = BM * 128;
  static constexpr bool kWgrad = MK == kOpKs;
  static constexpr int kLds = NSN * kNStage + NSM * kMStage;
  // loads that may be in flight at a point: those issued after the stage it waits for. A point
  // issues its m stage, then its n stage.
  static constexpr int kFlying = NSM == NSN ? (MQ + NQ) * (NSN - 2) : NQ;
  static_assert(kLds <= 160 * 1024, "LDS budget");
  static_assert(NQ * kThreads == BN * 8 && MQ * kThreads == BM * 8, "whole chunks");
  static_assert(NSN >= 2 && (NSM == NSN || (NSM == 2 && NSN == 3)), "ring depths");
  static_assert(kFlying < 64, "vmcnt range");
  using Acc = typename ProductTypes<EL>::Acc;

  // chunk `id` of a stage image in LDS order: the k row (strided) or row (contiguous) it belongs
  // to, and the logical chunk within that row whose place this is
  template <int KIND, int ROWS>
  static __device__ __forceinline__ void chunk_of(int id, int& row, int& c) {
    if constexpr (KIND == kOpKs) {
      constexpr int CPR = ROWS / 8;
      row = id / CPR;
      const int pc = id % CPR;
      c = ((((pc >> 1) ^ ks_swizzle<ROWS>(row)) << 1) | (pc & 1));
    } else {
      row = id >> 3;
      c = (id & 7) ^ kc_swizzle(row);
    }
  }

  struct Frags {
    u32x4_t a[NI], b[NJ];
  };

  // where a tile's operands lie: uniform bases, per-lane byte offsets, bytes and count of stages
  struct Source {
    const uint8_t *nb, *mb;
    size_t nstep, mstep;
    uint32_t noff[NQ], moff[MQ];
    int whole, stages, left;  // whole stages, all stages, elements of the partial one
  };

  static __device__ __forceinline__ void set_source(const ProductArgs& p, const TileAt& at,
                                                    Source& s) {
    const int tid = threadIdx.x;
    int k_lo = 0, k_hi = p.K;
    if constexpr (kWgrad) wgrad_rows(p, at.e, k_lo, k_hi);
    const int klen = __builtin_amdgcn_readfirstlane(k_hi - k_lo);
    s.whole = klen / BK;
    s.left = klen - s.whole * BK;
    s.stages = s.whole + (s.left ? 1 : 0);
    const uint8_t* nb = p.n_base + (size_t)at.e * p.n_estride;
    if constexpr (NK == kOpKs) {
      nb += (size_t)k_lo * p.n_pitch + (size_t)at.n0 * EB;
      s.nstep = (size_t)BK * p.n_pitch;
    } else if constexpr (NK == kOpPanel) {
      nb += (size_t)(at.n0 >> 4) * p.n_pitch;
      s.nstep = 2048;
    } else {
      nb += (size_t)at.n0 * p.n_pitch;
      s.nstep = 128;
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      int row, c;
      chunk_of<NK, BN>(q * kThreads + tid, row, c);
      if constexpr (NK == kOpKs) {
        s.noff[q] = (uint32_t)(row * (int)p.n_pitch + min(8 * c, p.N - at.n0 - 8) * EB);
      } else {
        const int r = min(row, p.N - 1 - at.n0);
        if constexpr (NK == kOpPanel)
          s.noff[q] = (uint32_t)((r >> 4) * (int)p.n_pitch + (r & 15) * 128 + 16 * c);
        else
          s.noff[q] = (uint32_t)(r * (int)p.n_pitch + 16 * c);
      }
    }
    const uint8_t* mb = p.m_base;
    s.mstep = 128;
    if constexpr (kWgrad) {
      mb += (size_t)k_lo * p.m_pitch + (size_t)at.row0 * EB;
      s.mstep = (size_t)BK * p.m_pitch;
    } else if (!p.row_src) {
      mb += (size_t)at.row0 * p.m_pitch;
    }
#pragma unroll
    for (int q = 0; q < MQ; ++q) {
      int row, c;
      chunk_of<MK, BM>(q * kThreads + tid, row, c);
      if constexpr (kWgrad) {
        s.moff[q] = (uint32_t)(row * (int)p.m_pitch + min(8 * c, p.M - at.row0 - 8) * EB);
      } else {
        const int r = min(at.row0 + row, at.row_end - 1);
        s.moff[q] = (uint32_t)((p.row_src ? source_row(p, r) : r - at.row0) *
                                   (uint32_t)p.m_pitch + 16 * c);
      }
    }
    s.nb = uniform_ptr(nb);
    s.mb = uniform_ptr(mb);
  }

  // Every tile of the calling workgroup. `next(at)` gives its tiles in turn (false: no more). The
  // loads of a tile's first stages go out before the stores of the tile before it.
  template <class Next>
  static __device__ __forceinline__ void run(const ProductArgs& p, uint8_t* lds, Next next) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / WM, wm = wave % WM;
    TileAt at;
    if (!next(at)) return;
    Source s;

    const uint32_t ring = __builtin_amdgcn_readfirstlane(lds_address(lds));
    auto nslot = [&](int j) { return (j % NSN) * kNStage; };
    auto mslot = [&](int j) { return NSN * kNStage + (j % NSM) * kMStage; };
    auto load_n = [&](int j, int q) {
      dma16_at(s.nb + (size_t)j * s.nstep, s.noff[q],
               ring + nslot(j) + (q * kWaves + wave) * 1024);
    };
    auto load_m = [&](int j, int q) {
      dma16_at(s.mb + (size_t)j * s.mstep, s.moff[q],
               ring + mslot(j) + (q * kWaves + wave) * 1024);
    };
    // the same for a stage that may be the partial one (chunks are whole or absent)
    auto load_n_any = [&](int j, int q) {
      int row, c;
      chunk_of<NK, BN>(q * kThreads + tid, row, c);
      const bool there = j < s.whole || NK == kOpPanel ||
                         (NK == kOpKs ? row < s.left : c * (16 / EB) < s.left);
      dma16_from(there ? s.nb + (size_t)j * s.nstep + s.noff[q] : kZeroChunk,
                 ring + nslot(j) + (q * kWaves + wave) * 1024);
    };
    auto load_m_any = [&](int j, int q) {
      int row, c;
      chunk_of<MK, BM>(q * kThreads + tid, row, c);
      const bool there = j < s.whole || EL == kPeI8 ||
                         (MK == kOpKs ? row < s.left : c * (16 / EB) < s.left);
      dma16_from(there ? s.mb + (size_t)j * s.mstep + s.moff[q] : kZeroChunk,
                 ring + mslot(j) + (q * kWaves + wave) * 1024);
    };

    // Lane addresses of the fragments: one per operand where the fragments are constant offsets
    // apart, one per fragment in registers where they are not (computing them again for every read
    // costs a wave issue slots that its MFMAs need).
    const int nfrag = fragment_base<NK, BN>(wn * TN, lane);
    const int mfrag = fragment_base<MK, BM>(wm * TM, lane);
    int nplace[NI], mplace[NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i) nplace[i] = fragment_place<NK>(nfrag, i);
#pragma unroll
    for (int i = 0; i < NJ; ++i) mplace[i] = fragment_place<MK>(mfrag, i);
    // fragment i of a step in the order of first use: a[0], every b, the other a
    auto read_one = [&](Frags& f, const uint8_t* ns, const uint8_t* ms, int t, int i) {
      if (i == 0 || i > NJ) {
        const int q = i == 0 ? 0 : i - NJ;
        if constexpr (NK == kOpKs) f.a[q] = read_place<NK, BN>(ns, nplace[q], t);
        else f.a[q] = read_fragment<NK, BN>(ns, nfrag, q, t);
      } else {
        if constexpr (MK == kOpKs) f.b[i - 1] = read_place<MK, BM>(ms, mplace[i - 1], t);
        else f.b[i - 1] = read_fragment<MK, BM>(ms, mfrag, i - 1, t);
      }
    };
    auto pin_places = [&]() {
#if defined(__HIP_DEVICE_COMPILE__)
      if constexpr (NK == kOpKs) {
#pragma unroll
        for (int i = 0; i < NI; ++i) asm volatile("" : "+v"(nplace[i]));
      }
      if constexpr (MK == kOpKs) {
#pragma unroll
        for (int i = 0; i < NJ; ++i) asm volatile("" : "+v"(mplace[i]));
      }
#endif
    };

    // Point j: the wait and barrier that make stage j readable, then its loads, m stage j + NSM - 1
    // and n stage j + NSN - 1: part 0 of them behind the barrier, in the last step of stage j - 1,
    // part 1 in the first step of stage j.
    constexpr int U = MQ + NQ;
    auto load_unit = [&](int j, int u) {  // unit u of point j's loads, whole stages
      if (u < MQ) load_m(j + NSM - 1, u);
      else load_n(j + NSN - 1, u - MQ);
    };
    auto load_part = [&](int j, int part) {  // part 0 or 1 of point j's loads, where they exist
#pragma unroll
      for (int u = part * U / 2; u < (part + 1) * U / 2; ++u) {
        if (u < MQ) {
          if (j + NSM - 1 < s.stages) load_m_any(j + NSM - 1, u);
        } else {
          if (j + NSN - 1 < s.stages) load_n_any(j + NSN - 1, u - MQ);
        }
      }
    };
    // (with NSM = 2, NSN = 3 the loads behind stage j's are those of n stage j + 1; with equal
    // depths those of stages j + 1 .. j + NSN - 2; where some of them do not exist, all are waited
    // for)
    auto point = [&](int j) {
      constexpr int LAST = NSM == NSN ? NSN - 2 : 1;
      if (j + LAST < s.stages) wait_vmcnt_fenced<kFlying>();
      else wait_vmcnt_fenced<0>();
      lds_barrier();
    };
    auto prologue = [&]() {  // the points before 0
#pragma unroll
      for (int j = 1 - NSN; j < 0; ++j) {
        if (j + NSM - 1 >= 0 && j + NSM - 1 < s.stages) {
#pragma unroll
          for (int q = 0; q < MQ; ++q) load_m_any(j + NSM - 1, q);
        }
        if (j + NSN - 1 < s.stages) {
#pragma unroll
          for (int q = 0; q < NQ; ++q) load_n_any(j + NSN - 1, q);
        }
      }
    };

    Acc acc[NI][NJ];
    // step t of stage j on fragments `cur`: its MFMAs with, between them, the reads of the next
    // step into `nxt` and a part of the loads of the current point
    constexpr int NM = NI * NJ, NR = NI + NJ;
    auto step = [&](int j, auto t_tag, auto steady, Frags& cur, Frags& nxt) {
      constexpr int t = decltype(t_tag)::value;
      constexpr bool S = decltype(steady)::value;
      constexpr bool LAST = t == 1;
      constexpr int PART = LAST ? 0 : 1;                // part of the point's loads sent here
      constexpr int D0 = PART * U / 2, ND = S ? (PART + 1) * U / 2 - D0 : 0;
      constexpr int OPS = NR + ND;
      constexpr int SLOTS = NM >= 16 ? NM * 3 / 4 : NM; // (the last MFMAs cover the last reads)
      const bool more = !LAST || j + 1 < s.stages;      // (STEADY: always)
      const uint8_t* ns = lds + nslot(LAST ? j + 1 : j);
      const uint8_t* ms = lds + mslot(LAST ? j + 1 : j);
      const int dj = LAST ? j + 1 : j;                  // whose point's loads go out here
#pragma unroll
      for (int i = 0; i < NM; ++i) acc_pin(acc[i / NJ][i % NJ]);
      if (!S && !LAST) load_part(j, 1);
      if (!S && LAST && more) {
        point(j + 1);
        load_part(j + 1, 0);
      }
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        acc[m / NJ][m % NJ] =
            product_mfma<EL>(cur.a[m / NJ], cur.b[m % NJ], acc[m / NJ][m % NJ]);
        __builtin_amdgcn_sched_barrier(0);
        if (S && LAST && m == 0) {
          wait_vmcnt_fenced<kFlying>();
          lds_barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
        if (!S && !more) continue;
#pragma unroll
        for (int op = m * OPS / SLOTS; op < (m + 1) * OPS / SLOTS; ++op) {
          // reads and loads in turn, the rest of the longer list last
          if (op < OPS) {
            constexpr int PAIRS = 2 * (ND < NR ? ND : NR);
            const bool load = op < PAIRS ? op % 2 == 1 : ND > NR;
            const int k = op < PAIRS ? op / 2 : op - PAIRS / 2;
            if (load) load_unit(dj, D0 + k);
            else read_one(nxt, ns, ms, LAST ? 0 : t + 1, k);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto stage = [&](int j, auto steady, Frags& f0, Frags& f1) {
      step(j, std::integral_constant<int, 0>{}, steady, f0, f1);
      step(j, std::integral_constant<int, 1>{}, steady, f1, f0);
    };

    set_source(p, at, s);
    prologue();
    while (true) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] = 0;
#pragma unroll
      for (int i = 0; i < NM; ++i) acc_pin(acc[i / NJ][i % NJ]);
      if (s.stages > 0) {
        Frags f0, f1;
        // everything is waited for here, the stores of the tile before included: they were issued
        // after this tile's first loads, and a count cannot tell which of the two has returned
        wait_vmcnt_fenced<0>();
        lds_barrier();
        load_part(0, 0);
#pragma unroll
        for (int i = 0; i < NR; ++i) read_one(f0, lds + nslot(0), lds + mslot(0), 0, i);
        int j = 0;
        for (; j + NSN < s.whole; ++j) {
          pin_places();
          stage(j, std::true_type{}, f0, f1);
        }
        for (; j < s.stages; ++j) stage(j, std::false_type{}, f0, f1);
      }
      const TileAt done = at;
      // int8: the scales of the finished tile, loaded before the next tile's stages
      float ms[NJ];
      f32x4v_t sc[NI], bs[NI];
      if constexpr (EL == kPeI8) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          ms[j] = p.m_scale[source_row(
              p, min(done.row0 + wm * TM + 16 * j + (lane & 15), done.row_end - 1))];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          // four columns' values; behind the last whole four of them one by one
          const int n = done.n0 + wn * TN + 16 * i + 4 * (lane >> 4);
          const size_t c = (size_t)done.e * p.N;
          auto four = [&](const float* f) {
            f32x4v_t v;
            if (n + 4 <= p.N) {
              v = *reinterpret_cast<const f32x4_any_t*>(f + c + n);
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = f[c + min(n + q, p.N - 1)];
            }
            return v;
          };
          sc[i] = four(p.n_scale);
          bs[i] = p.bias ? four(p.bias) : f32x4v_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
        for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(ms[j]));
#pragma unroll
        for (int i = 0; i < NI; ++i) asm volatile("" : "+v"(sc[i]), "+v"(bs[i]));
#endif
      }
      lds_barrier();  // every fragment of the tile is read: its ring slots are free
      const bool more = next(at);
      if (more) {
        set_source(p, at, s);
        prologue();
      }
      // The output, straight from the accumulators: acc[i][j][q] is column
      // n0 + wn TN + 16 i + 4 (lane / 16) + q of row row0 + wm TM + 16 j + lane % 16, so a store
      // writes 32 (16-bit) or 64 bytes of 16 rows. A whole tile's stores carry no conditions, and
      // each row of fragments is only taken out of its accumulators when it is stored.
      const int row_lim = kWgrad ? p.M : done.row_end;
      const int n = done.n0 + wn * TN + 4 * (lane >> 4);
      auto store = [&](auto kind_tag, auto whole_tag) {
        constexpr int KIND = decltype(kind_tag)::value;
        constexpr bool WHOLE = decltype(whole_tag)::value;
        constexpr int ES = KIND == kOutF32 ? 4 : 2;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
#pragma unroll
          for (int i = 0; i < NI; ++i) acc_pin(acc[i][j]);
          const int r = done.row0 + wm * TM + 16 * j + (lane & 15);
          if (!WHOLE && r >= row_lim) continue;
          uint8_t* o = reinterpret_cast<uint8_t*>(p.out) +
                       (((size_t)r + (kWgrad ? (size_t)done.e * p.M : 0)) * p.out_ld + n) * ES;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            if (!WHOLE && n + 16 * i >= p.N) continue;
            f32x4v_t v;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              v[q] = (float)acc[i][j][q];
              if constexpr (EL == kPeI8) v[q] = v[q] * ms[j] * sc[i][q];
            }
            if (EL == kPeI8 && p.bias) v += bs[i];
            if (!WHOLE) {
              store_run(p, (size_t)(o - reinterpret_cast<uint8_t*>(p.out)) / ES + 16 * i, n + 16 * i, v);
            } else if constexpr (KIND == kOutF32) {
              *reinterpret_cast<f32x4_any_t*>(o + 16 * i * ES) = v;
            } else {
              const uint2 b = KIND == kOutBf16 ? round_bf16x4(v) : round_fp16x4(v);
              *reinterpret_cast<u32x2_any_t*>(o + 16 * i * ES) = u32x2_any_t{b.x, b.y};
            }
          }
        }
      };
      auto store_kind = [&](auto whole_tag) {
        if (p.out_kind == kOutF32) store(std::integral_constant<int, kOutF32>{}, whole_tag);
        else if (p.out_kind == kOutBf16) store(std::integral_constant<int, kOutBf16>{}, whole_tag);
        else store(std::integral_constant<int, kOutFp16>{}, whole_tag);
      };
      if (done.n0 + BN <= p.N && done.row0 + BM <= row_lim) store_kind(std::true_type{});
      else store_kind(std::false_type{});
      if (!more) return;
    }
  }
};

}  // namespace
}  // namespace moe
