// Ragged grouped products: out[r] = rows[r] W[e(r)], the two gradients, and the int8 forms, with
// plain (unprepared) 16-bit weights in either order and any sizes.
//
// The tile kernel. A workgroup of four waves computes BN output columns x BM output rows, 128
// bytes of the sum index per stage: each thread loads its 16-byte chunks of the next stage into
// registers while the MFMAs run on the current one, and writes them to the other half of a
// double-buffered LDS image. Chunks that pass the end of a row, of the columns or of an expert's
// rows are zero in LDS, so every size is covered by the same loop and nothing that lies behind an
// expert's rows (another expert's infinities, unwritten memory) enters a sum.
#include "moe_product_big.h"

namespace moe {
namespace {

template <int EL, int NK, int MK, int BN, int BM, int WN>
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
    if constexpr (kWgrad) expert_rows(p, e, k_lo, k_hi);
    const int klen = k_hi - k_lo;
    const int stages = (klen + BK - 1) / BK;

    const uint8_t* nb = p.n_base + (size_t)e * p.n_estride;
    const uint8_t* nsrc[NQ];
    int nlim[NQ];  // contiguous: 1 if the row exists; strided: columns left from the chunk
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int id = q * 256 + tid;
      if constexpr (NK == kOpKs) {
        const int kk = id / (BN / 8), c = id % (BN / 8);
        nsrc[q] = nb + (size_t)(k_lo + kk) * p.n_pitch + (size_t)(n0 + 8 * c) * EB;
        nlim[q] = p.N - (n0 + 8 * c);
      } else if constexpr (NK == kOpPanel) {
        const int n = n0 + (id >> 3), c = id & 7;
        nsrc[q] = nb + (size_t)(n >> 4) * p.n_pitch + (n & 15) * 128 + 16 * c;
        nlim[q] = n < p.N;
      } else {
        const int n = n0 + (id >> 3), c = id & 7;
        nsrc[q] = nb + (size_t)n * p.n_pitch + 16 * c;
        nlim[q] = n < p.N;
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
        const int r = row0 + (id >> 3), c = id & 7;
        const bool ok = r < row_end;
        msrc[q] = p.m_base + (ok ? (size_t)source_row(p, r) * p.m_pitch : 0) + 16 * c;
        mlim[q] = ok;
      }
    }

    u32x4_t nreg[NQ], mreg[MQ];
    auto fetch = [&](int j) {  // stage j into registers
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int id = q * 256 + tid;
        if constexpr (NK == kOpKs) {
          const int kk = id / (BN / 8);
          const bool ok = j * BK + kk < klen;
          nreg[q] = load_chunk<EB>(nsrc[q] + (size_t)j * BK * p.n_pitch, ok ? nlim[q] : 0);
        } else if constexpr (NK == kOpPanel) {
          nreg[q] = load_chunk<EB>(nsrc[q] + (size_t)j * 2048, nlim[q] ? 16 : 0);
        } else {
          nreg[q] = load_chunk<EB>(nsrc[q] + (size_t)j * 128,
                                   nlim[q] ? klen - (j * BK + (id & 7) * (16 / EB)) : 0);
        }
      }
#pragma unroll
      for (int q = 0; q < MQ; ++q) {
        const int id = q * 256 + tid;
        if constexpr (MK == kOpKs) {
          const int kk = j * BK + id / (BM / 8);
          const bool ok = kk < klen;
          const size_t r = ok ? (size_t)source_row(p, k_lo + kk) : 0;
          mreg[q] = load_chunk<EB>(msrc[q] + r * p.m_pitch, ok ? mlim[q] : 0);
        } else if constexpr (EL == kPeI8) {  // code rows are padded to whole stages
          mreg[q] = load_chunk<EB>(msrc[q] + (size_t)j * 128, mlim[q] ? 16 : 0);
        } else {
          mreg[q] = load_chunk<EB>(msrc[q] + (size_t)j * 128,
                                   mlim[q] ? klen - (j * BK + (id & 7) * (16 / EB)) : 0);
        }
      }
    };
    auto put = [&](int b) {  // registers into LDS half b
      uint8_t* s = lds + b * kStage;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        *reinterpret_cast<u32x4_t*>(s + stage_byte<NK, BN>(q * 256 + tid)) = nreg[q];
#pragma unroll
      for (int q = 0; q < MQ; ++q)
        *reinterpret_cast<u32x4_t*>(s + BN * 128 + stage_byte<MK, BM>(q * 256 + tid)) = mreg[q];
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
    if (stages > 0) {
      fetch(0);
      put(0);
    }
    for (int j = 0; j < stages; ++j) {
      __syncthreads();
      if (j + 1 < stages) fetch(j + 1);
      const uint8_t* s = lds + (j & 1) * kStage;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4_t a[NI], b[NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i)
          a[i] = read_fragment<NK, BN>(s, nfrag, i, t);
#pragma unroll
        for (int i = 0; i < NJ; ++i)
          b[i] = read_fragment<MK, BM>(s + BN * 128, mfrag, i, t);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int q = 0; q < NJ; ++q) acc[i][q] = product_mfma<EL>(a[i], b[q], acc[i][q]);
      }
      if (j + 1 < stages) put((j + 1) & 1);
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
         big_tile_coords(mt * p.E, nt_total, p.band_gm, xcd, jx, ti, nt); jx += gridDim.x >> 3) {
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

template <int EL, int NK, int MK, int BN, int BM, int WN>
__global__ __launch_bounds__(256, 2) void product_tile_kernel(ProductArgs p) {
  using Tile = ProductTile<EL, NK, MK, BN, BM, WN>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Tile::kLds];
  __shared__ int scratch[4];
  product_tiles<Tile, BN, BM, 4>(p, lds, scratch);
}

template <int EL, int NK, int MK, int BN, int BM, int WN, int WM, int NSN, int NSM>
__global__ __launch_bounds__(64 * WN * WM, WN * WM / 4) void product_big_kernel(ProductArgs p) {
  using Tile = ProductBig<EL, NK, MK, BN, BM, WN, WM, NSN, NSM>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Tile::kLds];
  const int nt_total = (p.N + BN - 1) / BN;
  int jx = blockIdx.x >> 3;
  const int xcd = blockIdx.x & 7, per = gridDim.x >> 3;
  if constexpr (Tile::kWgrad) {
    const int mt = (p.M + BM - 1) / BM;
    Tile::run(p, lds, [&](TileAt& at) {
      int ti, nt;
      if (!big_tile_coords(mt * p.E, nt_total, p.band_gm, xcd, jx, ti, nt)) return false;
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

template <int EL, int NK, int MK, int BN, int BM, int WN>
hipError_t launch_tile(const ProductArgs& p, long long tiles, hipStream_t st) {
  hipLaunchKernelGGL((product_tile_kernel<EL, NK, MK, BN, BM, WN>), dim3(product_grid(tiles, 512)),
                     dim3(256), 0, st, p);
  return hipGetLastError();
}

template <int EL, int NK, int MK, int BN, int BM, int WN, int WM, int NSN, int NSM>
hipError_t launch_big(const ProductArgs& p, long long tiles, hipStream_t st) {
  hipLaunchKernelGGL((product_big_kernel<EL, NK, MK, BN, BM, WN, WM, NSN, NSM>),
                     dim3(product_grid(tiles, 256)), dim3(64 * WN * WM), 0, st, p);
  return hipGetLastError();
}

// M tiles of bm rows that R rows over E experts can need
long long row_tiles(const ProductArgs& p, int bm) {
  return (long long)(p.R / bm) + (p.E < p.R ? p.E : p.R);
}

// what the large tile's direct loads and stores need: rows at 16-byte steps, a sum (16-bit types)
// and contiguous columns of whole 16-byte chunks, gathered rows within 32-bit offsets, and output
// columns in whole runs of four
template <int NK>
bool big_rows_ok(const ProductArgs& p) {
  if (p.m_pitch % 16 || p.n_pitch % 16) return false;
  if (p.N % 4 || !p.out_vec) return false;
  if (NK != kOpPanel && p.K % 8) return false;
  if (NK == kOpKs && p.N % 8) return false;
  return !p.row_src || (unsigned long long)p.src_rows * p.m_pitch < (1ull << 32);
}

template <int EL, int NK>
hipError_t launch_rows(ProductArgs& p, hipStream_t st) {
  const long long rpe = (p.R + p.E - 1) / p.E;
  if (rpe > 64 && p.N >= 256 && big_rows_ok<NK>(p)) {
    const int bm = rpe >= 384 ? 256 : 128, nt = (p.N + 255) / 256;
    p.band_gm = band_groups_for(nt, bm, rpe);
    if (bm == 256) return launch_big<EL, NK, kOpKc, 256, 256, 2, 2, 3, 2>(p, row_tiles(p, bm) * nt, st);
    return launch_big<EL, NK, kOpKc, 256, 128, 2, 2, 3, 3>(p, row_tiles(p, bm) * nt, st);
  }
  const int bm = rpe <= 32 ? 32 : (rpe <= 64 ? 64 : 128);
  const int nt = (p.N + 127) / 128;
  p.band_gm = band_groups_for(nt, bm, rpe);
  const long long tiles = row_tiles(p, bm) * nt;
  if (bm == 32) return launch_tile<EL, NK, kOpKc, 128, 32, 4>(p, tiles, st);
  if (bm == 64) return launch_tile<EL, NK, kOpKc, 128, 64, 2>(p, tiles, st);
  return launch_tile<EL, NK, kOpKc, 128, 128, 2>(p, tiles, st);
}

template <int EL>
hipError_t launch_wgrad(ProductArgs& p, hipStream_t st) {
  if (p.m_pitch % 16 == 0 && p.n_pitch % 16 == 0 && p.M % 8 == 0 && p.N % 8 == 0 && !p.row_src &&
      p.M >= 256 && p.N >= 256) {
    const int nt = (p.N + 255) / 256, mt = (p.M + 255) / 256;
    p.band_gm = band_groups_for(nt, 256, p.M);
    return launch_big<EL, kOpKs, kOpKs, 256, 256, 2, 2, 3, 2>(p, (long long)mt * nt * p.E, st);
  }
  const int nt = (p.N + 127) / 128, mt = (p.M + 127) / 128;
  p.band_gm = band_groups_for(nt, 128, p.M);
  return launch_tile<EL, kOpKs, kOpKs, 128, 128, 2>(p, (long long)mt * nt * p.E, st);
}

}  // namespace

hipError_t launch_grouped_gemm(ProductArgs p, int el, bool trans_w, hipStream_t st) {
  if (el == kPeBf16)
    return trans_w ? launch_rows<kPeBf16, kOpKc>(p, st) : launch_rows<kPeBf16, kOpKs>(p, st);
  return trans_w ? launch_rows<kPeFp16, kOpKc>(p, st) : launch_rows<kPeFp16, kOpKs>(p, st);
}

hipError_t launch_grouped_wgrad(ProductArgs p, int el, hipStream_t st) {
  return el == kPeBf16 ? launch_wgrad<kPeBf16>(p, st) : launch_wgrad<kPeFp16>(p, st);
}

hipError_t launch_int8_gemm(ProductArgs p, hipStream_t st) {
  // Too few 128-column tiles to fill the CUs: split the sum over waves instead. The few-row kernel
  // reads the codes once per 16 columns, so its work grows with rows x columns: measured equal at
  // rows (each expert's at least 16) x 128-column tiles = 4096 (1 x 128 rows of 7168 x 4096: 37 us
  // against the tile's 57; 4 x 64 rows: 66 against 49; 8 x 1: 42 against 42), and for short sums,
  // where a tile's latency is short too, earlier (64 x 2 rows of 512 x 512: 13.5 against 6.4).
  const long long hit = p.E < p.R ? p.E : p.R, r16 = p.R > 16 * hit ? p.R : 16 * hit;
  const long long size = r16 * ((p.N + 127) / 128);
  if (size <= (p.K >= 2048 ? 4096 : 1024))
    return launch_int8_few(p, (p.R + p.E - 1) / p.E, st);
  return launch_rows<kPeI8, kOpPanel>(p, st);
}

}  // namespace moe
