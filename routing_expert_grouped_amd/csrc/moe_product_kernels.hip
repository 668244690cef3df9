// Ragged grouped products: out[r] = rows[r] W[e(r)], the two gradients, and the int8 forms, with
// plain (unprepared) 16-bit weights in either order and any sizes.
//
// The tile kernel. A workgroup of four waves computes BN output columns x BM output rows, 128
// bytes of the sum index per stage: each thread loads its 16-byte chunks of the next stage into
// registers while the MFMAs run on the current one, and writes them to the other half of a
// double-buffered LDS image. Chunks that pass the end of a row, of the columns or of an expert's
// rows are zero in LDS, so every size is covered by the same loop and nothing that lies behind an
// expert's rows (another expert's infinities, unwritten memory) enters a sum.
#include "moe_product.h"

namespace moe {
namespace {

template <int EL, int NK, int MK, int BN, int BM, int WN>
struct ProductTile {
  static constexpr int WM = 4 / WN;            // waves along the rows
  static constexpr int NI = BN / WN / 32;      // n fragments per wave
  static constexpr int NJ = BM / WM / 32;      // m fragments per wave
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
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;

    if (stages > 0) {
      fetch(0);
      put(0);
    }
    for (int j = 0; j < stages; ++j) {
      __syncthreads();
      if (j + 1 < stages) fetch(j + 1);
      const uint8_t* s = lds + (j & 1) * kStage;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        u32x4_t a[NI], b[NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i)
          a[i] = read_fragment<NK, BN>(s, wn * (BN / WN) + 32 * i, t, lane);
#pragma unroll
        for (int i = 0; i < NJ; ++i)
          b[i] = read_fragment<MK, BM>(s + BN * 128, wm * (BM / WM) + 32 * i, t, lane);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int q = 0; q < NJ; ++q) acc[i][q] = product_mfma<EL>(a[i], b[q], acc[i][q]);
      }
      if (j + 1 < stages) put((j + 1) & 1);
    }

    // acc[i][j][q]: column n0 + wn BN/WN + 32 i + 8 (q / 4) + 4 (lane / 32) + q % 4,
    //               row row0 + wm BM/WM + 32 j + lane % 32
    const int row_lim = kWgrad ? p.M : row_end;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int r = row0 + wm * (BM / WM) + 32 * j + (lane & 31);
      if (r >= row_lim) continue;
      const size_t at = ((size_t)r + (kWgrad ? (size_t)e * p.M : 0)) * p.out_ld;
      float ms = 0.0f;
      if constexpr (EL == kPeI8) ms = p.m_scale[source_row(p, r)];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int b4 = 0; b4 < 4; ++b4) {
          const int n = n0 + wn * (BN / WN) + 32 * i + 8 * b4 + 4 * (lane >> 5);
          if (n >= p.N) continue;
          f32x4v_t v;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[q] = (float)acc[i][j][4 * b4 + q];
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

template <int EL, int NK, int MK, int BN, int BM, int WN>
__global__ __launch_bounds__(256, 2) void product_tile_kernel(ProductArgs p) {
  using Tile = ProductTile<EL, NK, MK, BN, BM, WN>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Tile::kLds];
  __shared__ int scratch[4];
  const int nt_total = (p.N + BN - 1) / BN;
  if constexpr (Tile::kWgrad) {
    const int mt = (p.M + BM - 1) / BM;
    const int per = mt * nt_total;
    for (long long t = blockIdx.x; t < (long long)per * p.E; t += gridDim.x) {
      const int e = (int)(t / per), i = (int)(t % per);
      Tile::run(p, e, (i / nt_total) * BM, 0, (i % nt_total) * BN, lds);
      __syncthreads();
    }
  } else {
    const TileIndex x = tile_index(p, BM, scratch);
    const int xcd = blockIdx.x & 7;
    for (int jx = blockIdx.x >> 3;; jx += gridDim.x >> 3) {
      int ti, nt;
      if (!big_tile_coords(x.total, nt_total, p.band_gm, xcd, jx, ti, nt)) break;
      int e, row0, row_end;
      tile_lookup(p, x, ti, BM, scratch, e, row0, row_end);
      Tile::run(p, e, row0, row_end, nt * BN, lds);
      __syncthreads();
    }
  }
}

// workgroups of a persistent launch: at most two per CU of the device, no more than the tiles
// there can be, and a multiple of 8 (one share per XCD)
unsigned product_grid(long long tiles) {
  const long long g = tiles < 512 ? tiles : 512;
  return (unsigned)((g + 7) / 8 * 8);
}

template <int EL, int NK, int MK, int BN, int BM, int WN>
hipError_t launch_tile(const ProductArgs& p, long long tiles, hipStream_t st) {
  hipLaunchKernelGGL((product_tile_kernel<EL, NK, MK, BN, BM, WN>), dim3(product_grid(tiles)),
                     dim3(256), 0, st, p);
  return hipGetLastError();
}

template <int EL, int NK>
hipError_t launch_rows(ProductArgs& p, hipStream_t st) {
  const long long rpe = (p.R + p.E - 1) / p.E;
  const int bm = rpe <= 32 ? 32 : (rpe <= 64 ? 64 : 128);
  const int nt = (p.N + 127) / 128;
  const long long mt = (long long)(p.R / bm) + (p.E < p.R ? p.E : p.R);
  p.band_gm = band_groups_for(nt, bm, rpe);
  if (bm == 32) return launch_tile<EL, NK, kOpKc, 128, 32, 4>(p, mt * nt, st);
  if (bm == 64) return launch_tile<EL, NK, kOpKc, 128, 64, 2>(p, mt * nt, st);
  return launch_tile<EL, NK, kOpKc, 128, 128, 2>(p, mt * nt, st);
}

}  // namespace

hipError_t launch_grouped_gemm(ProductArgs p, int el, bool trans_w, hipStream_t st) {
  if (el == kPeBf16)
    return trans_w ? launch_rows<kPeBf16, kOpKc>(p, st) : launch_rows<kPeBf16, kOpKs>(p, st);
  return trans_w ? launch_rows<kPeFp16, kOpKc>(p, st) : launch_rows<kPeFp16, kOpKs>(p, st);
}

hipError_t launch_grouped_wgrad(ProductArgs p, int el, hipStream_t st) {
  const long long tiles = (long long)((p.M + 127) / 128) * ((p.N + 127) / 128) * p.E;
  if (el == kPeBf16) return launch_tile<kPeBf16, kOpKs, kOpKs, 128, 128, 2>(p, tiles, st);
  return launch_tile<kPeFp16, kOpKs, kOpKs, 128, 128, 2>(p, tiles, st);
}

hipError_t launch_int8_gemm(ProductArgs p, hipStream_t st) {
  return launch_rows<kPeI8, kOpPanel>(p, st);
}

}  // namespace moe
