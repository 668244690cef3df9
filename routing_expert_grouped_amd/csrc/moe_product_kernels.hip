// Ragged grouped products: out[r] = rows[r] W[e(r)], the two gradients, and the int8 forms, with
// plain (unprepared) 16-bit weights in either order and any sizes.
//
// Two families of tiles. ProductBig (moe_product_big.h) brings its operands to LDS by direct loads
// and takes what those can address; ProductTile below takes everything else: row pitches that are no
// multiple of 16 bytes, sums (or columns of a strided operand) that are no whole chunks, gathered
// weight gradients. A thread loads its 16-byte chunks of the stages ahead into registers while the
// MFMAs run, and writes them to the other half of a double-buffered LDS image. In the stage that
// passes the end of the sum, what lies behind it is zero in LDS, so nothing there (another expert's
// infinities, unwritten memory) enters a sum; rows and columns behind the tile's edge repeat its
// last ones and are not stored. Loads carry no branches (a chunk that passes its row's end is
// loaded from the row's last eight elements and shifted), or the compiler would wait for each
// before the next.
// Measured, 8192 x 4095 x 4095 bf16: forward 508, input gradient 685, weight gradient 522 TFLOP/s.
//
// Which tile a call takes is estimated from its rounds over the CUs (launch_rows). Measured at two
// sides of it: 4299 rows, 1244 x 1552 int8 over 3 experts, take 36 us with 126 tiles of 256 x 256 and
// 26 with twice as many of 256 x 128 (half the CUs against all); 11076 rows, 5248 x 640 bf16 over 15
// experts, take 136 us with some 150 tiles of 256 x 256 and 152 with 256 x 128 (one round against
// two).
#include "moe_product_big.h"

namespace moe {
namespace {

// PF: stages in registers ahead of the one in LDS. TINY: an operand's rows are shorter than a chunk
// (8 elements), everything is loaded element by element.
template <int EL, int NK, int MK, int BN, int BM, int WN, int PF, bool TINY>
struct ProductTile {
  static constexpr int WM = 4 / WN;            // waves along the rows
  static constexpr int NI = BN / WN / 16;      // n fragments per wave
  static constexpr int NJ = BM / WM / 16;      // m fragments per wave
  static constexpr int NQ = BN * 8 / 256;      // 16-byte chunks per thread and stage, n operand
  static constexpr int MQ = BM * 8 / 256;
  static constexpr int EB = ProductTypes<EL>::kBytes;
  static constexpr int BK = 128 / EB;          // sum elements per stage
  static constexpr int kStage = (BN + BM) * 128;
  static constexpr int kLds = 2 * kStage;
  static constexpr bool kWgrad = MK == kOpKs;
  using Acc = typename ProductTypes<EL>::Acc;

  // one output tile; the caller separates two tiles by a barrier
  static __device__ __forceinline__ void run(const ProductArgs& p, int e, int row0, int row_end,
                                             int n0, uint8_t* lds) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / WM, wm = wave % WM;
    // the sum index: K columns, or the expert's rows
    int k_lo = 0, k_hi = p.K;
    if constexpr (kWgrad) wgrad_rows(p, e, k_lo, k_hi);
    const int klen = k_hi - k_lo;
    const int stages = (klen + BK - 1) / BK;

    const uint8_t* nb = p.n_base + (size_t)e * p.n_estride;
    const uint8_t* nsrc[NQ];
    int nlim[NQ];  // strided: columns left from the chunk
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int id = q * 256 + tid;
      if constexpr (NK == kOpKs) {
        const int kk = id / (BN / 8), c = id % (BN / 8);
        nsrc[q] = nb + (size_t)(k_lo + kk) * p.n_pitch + (size_t)(n0 + 8 * c) * EB;
        nlim[q] = p.N - (n0 + 8 * c);
      } else {
        const int n = min(n0 + (id >> 3), p.N - 1), c = id & 7;
        nsrc[q] = NK == kOpPanel
                      ? nb + (size_t)(n >> 4) * p.n_pitch + (n & 15) * 128 + 16 * c
                      : nb + (size_t)n * p.n_pitch + 16 * c;
      }
    }
    const uint8_t* msrc[MQ];
    int mlim[MQ];
#pragma unroll
    for (int q = 0; q < MQ; ++q) {
      const int id = q * 256 + tid;
      if constexpr (MK == kOpKs) {
        const int c = id % (BM / 8);
        msrc[q] = p.m_base + (size_t)(row0 + 8 * c) * EB;
        mlim[q] = p.M - (row0 + 8 * c);
      } else {
        const int r = min(row0 + (id >> 3), row_end - 1), c = id & 7;
        msrc[q] = p.m_base + (size_t)source_row(p, r) * p.m_pitch + 16 * c;
      }
    }

    struct Chunks {
      u32x4_t n[NQ], m[MQ];
    };
    // Elements of thread chunk q of stage j that exist, and (uniform) whether every chunk of the
    // stage may be taken as it lies: not past the end of the sum, nor, strided, in a tile whose
    // last columns are no whole chunk. (Code rows and panels are padded to whole stages.)
    auto n_valid = [&](int j, int q) {
      const int id = q * 256 + tid;
      if constexpr (NK == kOpKs) return j * BK + id / (BN / 8) < klen ? nlim[q] : 0;
      else return klen - (j * BK + (id & 7) * (16 / EB));
    };
    auto m_valid = [&](int j, int q) {
      const int id = q * 256 + tid;
      if constexpr (MK == kOpKs) return j * BK + id / (BM / 8) < klen ? mlim[q] : 0;
      else return klen - (j * BK + (id & 7) * (16 / EB));
    };
    const bool n_even = !TINY && (NK != kOpKs || n0 + BN <= p.N);
    const bool m_even = !TINY && (MK != kOpKs || row0 + BM <= p.M);
    auto exact = [&](int j, bool even) {
      return EL == kPeI8 || (even && (j + 1) * BK <= klen);
    };
    auto load = [&](bool whole, const uint8_t* at, int valid, const uint8_t* any) {
      if (whole) return *reinterpret_cast<const u32x4_any_t*>(at);
      if constexpr (TINY) return load_chunk<EB>(at, valid);
      else return load_chunk_raw(at, valid, any);
    };
    auto fetch = [&](int j, Chunks& x) {  // stage j's loads into registers
      const size_t step = NK == kOpKs ? BK * p.n_pitch : NK == kOpPanel ? 2048 : 128;
      const bool ne = exact(j, n_even), me = exact(j, m_even);
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        x.n[q] = load(ne, nsrc[q] + (size_t)j * step, n_valid(j, q), nb);
#pragma unroll
      for (int q = 0; q < MQ; ++q) {
        size_t at = (size_t)j * 128;
        if constexpr (MK == kOpKs) {
          const int kk = j * BK + (q * 256 + tid) / (BM / 8);
          at = (size_t)source_row(p, k_lo + min(kk, klen - 1)) * p.m_pitch;
        }
        x.m[q] = load(me, msrc[q] + at, m_valid(j, q), p.m_base);
      }
    };
    auto put = [&](int j, const Chunks& x) {  // stage j's registers into LDS half j % 2
      uint8_t* s = lds + (j & 1) * kStage;
      const bool ne = TINY || exact(j, n_even), me = TINY || exact(j, m_even);
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        *reinterpret_cast<u32x4_t*>(s + stage_byte<NK, BN>(q * 256 + tid)) =
            ne ? x.n[q] : settle_chunk(x.n[q], n_valid(j, q));
#pragma unroll
      for (int q = 0; q < MQ; ++q)
        *reinterpret_cast<u32x4_t*>(s + BN * 128 + stage_byte<MK, BM>(q * 256 + tid)) =
            me ? x.m[q] : settle_chunk(x.m[q], m_valid(j, q));
    };

    Acc acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = 0;

    const int nfrag = fragment_base<NK, BN>(wn * (BN / WN), lane);
    const int mfrag = fragment_base<MK, BM>(wm * (BM / WM), lane);
    // stage j from LDS half j % 2, `next` holding stage j + 1 and being refilled with j + 1 + PF
    auto stage = [&](int j, Chunks& next, Chunks& far) {
      __syncthreads();
      // (no condition: behind a branch the compiler would wait for these loads before it uses the
      // ones in front of them; past the end the last stage is loaded again and not used)
      fetch(min(j + PF, stages - 1), PF == 1 ? next : far);
      const uint8_t* s = lds + (j & 1) * kStage;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4_t a[NI], b[NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i) a[i] = read_fragment<NK, BN>(s, nfrag, i, t);
#pragma unroll
        for (int i = 0; i < NJ; ++i) b[i] = read_fragment<MK, BM>(s + BN * 128, mfrag, i, t);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int q = 0; q < NJ; ++q) acc[i][q] = product_mfma<EL>(a[i], b[q], acc[i][q]);
      }
      if (j + 1 < stages) put(j + 1, next);
    };
    Chunks x0, x1;
    if (stages > 0) {
      fetch(0, x0);
      if (PF == 2) fetch(min(1, stages - 1), x1);
      put(0, x0);
    }
    if constexpr (PF == 1) {
      for (int j = 0; j < stages; ++j) stage(j, x0, x0);
    } else {  // stage j + 1 waits in x1 for even j, in x0 for odd j
      int j = 0;
      for (; j + 1 < stages; j += 2) {
        stage(j, x1, x0);
        stage(j + 1, x0, x1);
      }
      if (j < stages) stage(j, x1, x0);
    }

    // acc[i][j][q]: column n0 + wn BN/WN + 16 i + 4 (lane / 16) + q,
    //               row row0 + wm BM/WM + 16 j + lane % 16
    const int row_lim = kWgrad ? p.M : row_end;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int r = row0 + wm * (BM / WM) + 16 * j + (lane & 15);
      if (r >= row_lim) continue;
      const size_t at = ((size_t)r + (kWgrad ? (size_t)e * p.M : 0)) * p.out_ld;
      float ms = 0.0f;
      if constexpr (EL == kPeI8) ms = p.m_scale[source_row(p, r)];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int n = n0 + wn * (BN / WN) + 16 * i + 4 * (lane >> 4);
        if (n >= p.N) continue;
        f32x4v_t v;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] = (float)acc[i][j][q];
          if constexpr (EL == kPeI8) {
            const size_t c = (size_t)e * p.N + min(n + q, p.N - 1);
            v[q] = v[q] * ms * p.n_scale[c];
            if (p.bias) v[q] += p.bias[c];
          }
        }
        store_run(p, at + n, n, v);
      }
    }
  }
};

// The tiles of one workgroup: a fixed share of its XCD's part of the tile order (big_tile_coords).
template <class Tile, int BN, int BM, int WAVES>
__device__ __forceinline__ void product_tiles(const ProductArgs& p, uint8_t* lds, int* scratch) {
  const int nt_total = (p.N + BN - 1) / BN;
  const int xcd = blockIdx.x & 7;
  int ti, nt;
  if constexpr (Tile::kWgrad) {
    const int mt = (p.M + BM - 1) / BM;
    for (int jx = blockIdx.x >> 3;
         big_tile_coords(mt * p.E * p.split, nt_total, p.band_gm, xcd, jx, ti, nt);
         jx += gridDim.x >> 3) {
      Tile::run(p, ti / mt, (ti % mt) * BM, 0, nt * BN, lds);
      __syncthreads();
    }
  } else {
    const TileIndex x = tile_index<WAVES>(p, BM, scratch);
    for (int jx = blockIdx.x >> 3; big_tile_coords(x.total, nt_total, p.band_gm, xcd, jx, ti, nt);
         jx += gridDim.x >> 3) {
      int e, row0, row_end;
      tile_lookup(p, x, ti, BM, scratch, e, row0, row_end);
      Tile::run(p, e, row0, row_end, nt * BN, lds);
      __syncthreads();
    }
  }
}

template <int EL, int NK, int MK, int BN, int BM, int WN, int PF, bool TINY>
__global__ __launch_bounds__(256, 2) void product_tile_kernel(ProductArgs p) {
  using Tile = ProductTile<EL, NK, MK, BN, BM, WN, PF, TINY>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Tile::kLds];
  __shared__ int scratch[4];
  product_tiles<Tile, BN, BM, 4>(p, lds, scratch);
}

// OCC: workgroups per CU
template <int EL, int NK, int MK, int BN, int BM, int WN, int WM, int NSN, int NSM, int OCC>
__global__ __launch_bounds__(64 * WN * WM, OCC * WN * WM / 4) void product_big_kernel(ProductArgs p) {
  using Tile = ProductBig<EL, NK, MK, BN, BM, WN, WM, NSN, NSM>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Tile::kLds];
  const int nt_total = (p.N + BN - 1) / BN;
  int jx = blockIdx.x >> 3;
  const int xcd = blockIdx.x & 7, per = gridDim.x >> 3;
  if constexpr (Tile::kWgrad) {
    const int mt = (p.M + BM - 1) / BM;
    Tile::run(p, lds, [&](TileAt& at) {
      int ti, nt;
      if (!big_tile_coords(mt * p.E * p.split, nt_total, p.band_gm, xcd, jx, ti, nt)) return false;
      jx += per;
      at.e = __builtin_amdgcn_readfirstlane(ti / mt);
      at.row0 = __builtin_amdgcn_readfirstlane((ti % mt) * BM);
      at.row_end = p.M;
      at.n0 = nt * BN;
      return true;
    });
  } else {
    const WaveTiles x = wave_tiles(p, BM);
    Tile::run(p, lds, [&](TileAt& at) {
      int ti, nt;
      if (!big_tile_coords(x.total, nt_total, p.band_gm, xcd, jx, ti, nt)) return false;
      jx += per;
      wave_lookup(p, x, __builtin_amdgcn_readfirstlane(ti), BM, at);
      at.n0 = __builtin_amdgcn_readfirstlane(nt * BN);
      return true;
    });
  }
}

// workgroups of a persistent launch: at most `slots` (those that run at once), no more than the
// tiles there can be, and a multiple of 8 (one share per XCD)
unsigned product_grid(long long tiles, long long slots) {
  const long long g = tiles < slots ? tiles : slots;
  return (unsigned)((g + 7) / 8 * 8);
}

template <int EL, int NK, int MK, int BN, int BM, int WN, int PF>
hipError_t launch_tile(const ProductArgs& p, long long tiles, hipStream_t st) {
  const dim3 g(product_grid(tiles, 512)), b(256);
  const bool tiny = EL != kPeI8 && ((NK == kOpKs ? p.N : p.K) < 8 || (MK == kOpKs ? p.M : p.K) < 8);
  if constexpr (BM <= 64 && EL != kPeI8) {
    if (tiny) {
      hipLaunchKernelGGL((product_tile_kernel<EL, NK, MK, BN, BM, WN, PF, true>), g, b, 0, st, p);
      return hipGetLastError();
    }
  }
  if (tiny) return hipErrorInvalidValue;  // (the callers send tiny rows to the 64-row tile)
  hipLaunchKernelGGL((product_tile_kernel<EL, NK, MK, BN, BM, WN, PF, false>), g, b, 0, st, p);
  return hipGetLastError();
}

template <int EL, int NK, int MK, int BN, int BM, int WN, int WM, int NSN, int NSM, int OCC>
hipError_t launch_big(const ProductArgs& p, long long tiles, hipStream_t st) {
  hipLaunchKernelGGL((product_big_kernel<EL, NK, MK, BN, BM, WN, WM, NSN, NSM, OCC>),
                     dim3(product_grid(tiles, 256 * OCC)), dim3(64 * WN * WM), 0, st, p);
  return hipGetLastError();
}

// M tiles of bm rows that R rows over E experts can need, and (for the choice of a tile) that they
// need when the last tile of an expert is half full
long long row_tiles(const ProductArgs& p, int bm) {
  return (long long)(p.R / bm) + (p.E < p.R ? p.E : p.R);
}
long long likely_row_tiles(const ProductArgs& p, int bm) {
  if (p.E == 1) return (p.R + bm - 1) / bm;
  return (long long)(p.R / bm) + ((p.E < p.R ? p.E : p.R) + 1) / 2;
}

// Relative time of `tiles` tiles of which `slots` run at once, each round taking `unit`. Units, in
// rounds of the 256 x 256 tile (8192 x 4096 x 4096 and the sizes around it, measured): 256 x 128
// runs at 0.87 of its rate, 0.57; two 64 x 64 tiles per CU at about half of it, 0.25; of the
// register-staged tiles 128 x 128 takes 2.7 rounds of 64 x 64.
double tile_cost(long long tiles, int slots, double unit) {
  return (double)((tiles + slots - 1) / slots) * unit;
}

// what the direct loads need of both operands: rows at 16-byte steps, and a tile's at most 256 of
// them within 32-bit offsets
bool pitches_ok(const ProductArgs& p) {
  return p.m_pitch % 16 == 0 && p.n_pitch % 16 == 0 && p.m_pitch <= (1u << 22) &&
         p.n_pitch <= (1u << 22);
}

// and of a product over routed rows: a sum (16-bit types) and contiguous columns of whole 16-byte
// chunks, and gathered rows within 32-bit offsets
template <int NK>
bool big_rows_ok(const ProductArgs& p) {
  if (!pitches_ok(p)) return false;
  if (NK != kOpPanel && p.K % 8) return false;
  if (NK == kOpKs && p.N % 8) return false;
  return !p.row_src || (unsigned long long)p.src_rows * p.m_pitch < (1ull << 32);
}

// The tile of a product over routed rows: the one whose rounds over the CUs are estimated cheapest
// (a large tile has the higher rate, a small one fills the CUs and wastes less at an expert's
// end), and 32 rows of 128 columns where an expert has at most 32 on average: reading the weights is
// all there is, and this tile has the most loads in flight for them. Unless there are so few of
// those that most CUs would idle: then 64 x 64 (bf16, 16 rows each, us: 32 tiles, 7168 x 4096, 48
// against 37; 128 tiles, 8 experts of 4096 x 2048, 25 against 24; 256 tiles, 16 of them, 43
// against 47).
template <int EL, int NK>
hipError_t launch_rows(ProductArgs& p, hipStream_t st) {
  const long long rpe = (p.R + p.E - 1) / p.E;
  const int n256 = (p.N + 255) / 256, n128 = (p.N + 127) / 128, n64 = (p.N + 63) / 64;
  const double c64 = tile_cost(likely_row_tiles(p, 64) * n64, 512, 0.25);
  const bool direct = big_rows_ok<NK>(p);
  const long long hit = p.E < p.R ? p.E : p.R;
  if (rpe <= 32 && !(direct && hit * n128 <= 128)) {
    const long long tiles = row_tiles(p, 32) * n128;
    p.band_gm = band_groups_for(n128, 32, rpe);
    if (direct) return launch_big<EL, NK, kOpKc, 128, 32, 4, 1, 4, 4, 2>(p, tiles, st);
    return launch_tile<EL, NK, kOpKc, 128, 32, 4, 2>(p, tiles, st);
  }
  if (direct) {
    const double c256 = tile_cost(likely_row_tiles(p, 256) * n256, 256, 1.0);
    const double c128 = tile_cost(likely_row_tiles(p, 128) * n256, 256, 0.57);
    if (c256 <= c128 && c256 <= c64) {
      p.band_gm = band_groups_for(n256, 256, rpe);
      return launch_big<EL, NK, kOpKc, 256, 256, 2, 2, 3, 2, 1>(p, row_tiles(p, 256) * n256, st);
    }
    if (c128 <= c64) {
      p.band_gm = band_groups_for(n256, 128, rpe);
      return launch_big<EL, NK, kOpKc, 256, 128, 2, 2, 3, 3, 1>(p, row_tiles(p, 128) * n256, st);
    }
    p.band_gm = band_groups_for(n64, 64, rpe);
    return launch_big<EL, NK, kOpKc, 64, 64, 2, 2, 4, 4, 2>(p, row_tiles(p, 64) * n64, st);
  }
  if (p.K >= 8 && p.N >= 8 &&
      tile_cost(likely_row_tiles(p, 128) * n128, 512, 2.7) <=
          tile_cost(likely_row_tiles(p, 64) * n64, 512, 1.0)) {
    p.band_gm = band_groups_for(n128, 128, rpe);
    return launch_tile<EL, NK, kOpKc, 128, 128, 2, 1>(p, row_tiles(p, 128) * n128, st);
  }
  p.band_gm = band_groups_for(n64, 64, rpe);
  return launch_tile<EL, NK, kOpKc, 64, 64, 2, 2>(p, row_tiles(p, 64) * n64, st);
}

// dw = the split parts added in order; four elements per thread
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* __restrict__ part, int split,
                                                         size_t count, void* __restrict__ out,
                                                         int out_kind) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  f32x4v_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool whole = count % 4 == 0;  // (then every part starts at a 16-byte step)
  for (int k = 0; k < split; ++k) {
    const float* q = part + (size_t)k * count + i;
    if (whole) {
      s += *reinterpret_cast<const f32x4v_t*>(q);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < count) s[j] += q[j];
    }
  }
  ProductArgs p{};  // (store_run's row: the rest of the array)
  p.out = out;
  p.out_kind = out_kind;
  p.N = count - i < 4 ? (int)(count - i) : 4;
  store_run(p, i, 0, s);
}

long long wgrad_tiles(int M, int N, int E, int b) {
  return (long long)((M + b - 1) / b) * ((N + b - 1) / b) * E;
}

template <int EL>
hipError_t launch_wgrad(ProductArgs& p, float* ws, hipStream_t st) {
  auto tiles = [&](int b) { return wgrad_tiles(p.M, p.N, p.E, b); };
  auto band = [&](int b) { return band_groups_for((p.N + b - 1) / b, b, p.M); };
  const long long t256 = tiles(256), t128 = tiles(128), t64 = tiles(64);
  const bool direct = pitches_ok(p) && p.M % 8 == 0 && p.N % 8 == 0 && !p.row_src;
  const int split = wgrad_split(p.M, p.N, p.E, p.R);
  if (split > 1) {  // into parts [split][E][M][N], then their sum
    ProductArgs q = p;
    q.split = split;
    q.out = ws;
    q.out_kind = kOutF32;
    q.band_gm = band(64);
    const hipError_t e =
        direct ? launch_big<EL, kOpKs, kOpKs, 64, 64, 2, 2, 4, 4, 2>(q, t64 * split, st)
               : launch_tile<EL, kOpKs, kOpKs, 64, 64, 2, 2>(q, t64 * split, st);
    if (e != hipSuccess) return e;
    const size_t count = (size_t)p.E * p.M * p.N;
    hipLaunchKernelGGL(wgrad_join_kernel, dim3((unsigned)((count + 1023) / 1024)), dim3(256), 0,
                       st, ws, split, count, p.out, p.out_kind);
    return hipGetLastError();
  }
  if (direct) {
    if (tile_cost(t256, 256, 1.0) <= tile_cost(t64, 512, 0.25)) {
      p.band_gm = band(256);
      return launch_big<EL, kOpKs, kOpKs, 256, 256, 2, 2, 3, 2, 1>(p, t256, st);
    }
    p.band_gm = band(64);
    return launch_big<EL, kOpKs, kOpKs, 64, 64, 2, 2, 4, 4, 2>(p, t64, st);
  }
  if (p.M >= 8 && p.N >= 8 && tile_cost(t128, 512, 2.7) <= tile_cost(t64, 512, 1.0)) {
    p.band_gm = band(128);
    return launch_tile<EL, kOpKs, kOpKs, 128, 128, 2, 1>(p, t128, st);
  }
  p.band_gm = band(64);
  return launch_tile<EL, kOpKs, kOpKs, 64, 64, 2, 2>(p, t64, st);
}

}  // namespace

hipError_t launch_grouped_gemm(ProductArgs p, int el, bool trans_w, hipStream_t st) {
  if (el == kPeBf16)
    return trans_w ? launch_rows<kPeBf16, kOpKc>(p, st) : launch_rows<kPeBf16, kOpKs>(p, st);
  return trans_w ? launch_rows<kPeFp16, kOpKc>(p, st) : launch_rows<kPeFp16, kOpKs>(p, st);
}

// Parts the rows of each expert are split into: where the 64 x 64 tiles of a small gradient do not
// fill the 512 places, as many as do, of at least 256 rows on average (what a part costs in
// writing and adding), at most 32.
int wgrad_split(int M, int N, int E, int R) {
  const long long t64 = wgrad_tiles(M, N, E, 64);
  long long s = 512 / t64;
  const long long rows = R / (256ll * E);
  s = s < rows ? s : rows;
  return (int)(s < 1 ? 1 : s > 32 ? 32 : s);
}

hipError_t launch_grouped_wgrad(ProductArgs p, int el, float* ws, hipStream_t st) {
  p.split = 1;
  return el == kPeBf16 ? launch_wgrad<kPeBf16>(p, ws, st) : launch_wgrad<kPeFp16>(p, ws, st);
}

hipError_t launch_int8_gemm(ProductArgs p, hipStream_t st) {
  // Few rows and too few tiles of 128 columns to fill the CUs: split the sum over waves instead.
  // Measured against the tiles, us. 32 tiles: 1 row of 7168 x 4096 10.1 / 17.8, 32 rows 16.0 / 18.6,
  // of 512 x 512 4.9 / 5.2. 64 tiles: 16 rows of 7168 x 8192 20.3 / 22.3, 32 rows 26.5 / 22.8, 16
  // rows of 2048 x 8192 8.3 / 7.5.
  const long long tiles = (long long)(p.E < p.R ? p.E : p.R) * ((p.N + 127) / 128);
  const int rpe = (p.R + p.E - 1) / p.E;
  if ((rpe <= 32 && tiles <= 32) || (p.R <= 16 && tiles <= 64 && p.K >= 4096))
    return launch_int8_few(p, rpe, st);
  return launch_rows<kPeI8, kOpPanel>(p, st);
}

}  // namespace moe
