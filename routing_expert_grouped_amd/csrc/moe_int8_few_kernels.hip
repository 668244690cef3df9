// The int8 product for few rows per expert: bound by reading the packed weights once.
//
// A workgroup of eight waves computes 16 output columns (one weight panel) x 16 NJ rows. The waves
// split the sum: wave w takes the panel's 2 KB blocks w, w + 8, ..., so the workgroup streams 16 KB
// in a row, straight into MFMA operands (a 16-row x 64-byte fragment is one 16-byte load per lane
// and the two fragments of a block are all of its 16 lines); the code rows come from the caches.
// Four blocks per wave are in flight at once. The waves' sums are integers, so adding them through
// LDS is exact in any order. Splitting over waves instead of columns keeps 256 workgroups busy on a
// 4096-column product of one token, where a tile of 128 columns would fill 32 CUs.
//
// Measured, 7168 x 4096 (29.4 MB of weights from memory): 1 row 10.1 us (2.9 TB/s), 16 rows 12.7,
// 32 rows 16.0 (the tiles: 21.7, 22.9, 24.7).
#include "moe_product.h"

namespace moe {
namespace {

constexpr int kFewWaves = 8;
constexpr int kFewUnroll = 4;  // blocks of a wave that are in flight at once
template <int NJ>
__global__ __launch_bounds__(64 * kFewWaves, 4) void int8_few_kernel(ProductArgs p) {
  __shared__ i32x4v_t part[kFewWaves][NJ][64];
  __shared__ int scratch[kFewWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int panels = (p.N + 15) / 16, blocks = (p.K + 127) / 128;
  const TileIndex x = tile_index<kFewWaves>(p, 16 * NJ, scratch);
  const int xcd = blockIdx.x & 7;
  const int koff = 16 * (lane >> 4);
  for (int jx = blockIdx.x >> 3;; jx += gridDim.x >> 3) {
    int ti, nt;
    if (!big_tile_coords(x.total, panels, p.band_gm, xcd, jx, ti, nt)) break;
    int e, row0, row_end;
    tile_lookup(p, x, ti, 16 * NJ, scratch, e, row0, row_end);
    const uint8_t* wp = p.n_base + (size_t)e * p.n_estride + (size_t)nt * p.n_pitch +
                        (lane & 15) * 128 + koff;
    const uint8_t* cp[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int r = min(row0 + 16 * j + (lane & 15), row_end - 1);  // (rows behind: not stored)
      cp[j] = p.m_base + (size_t)source_row(p, r) * p.m_pitch + koff;
    }
    i32x4v_t acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = i32x4v_t{0, 0, 0, 0};
    auto step = [&](int b0, auto count) {  // blocks b0, b0 + kFewWaves, ...
      constexpr int C = decltype(count)::value;
      u32x4_t w[C][2], c[C][NJ][2];
#pragma unroll
      for (int u = 0; u < C; ++u) {
        const size_t b = b0 + u * kFewWaves;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          w[u][t] = *reinterpret_cast<const u32x4_t*>(wp + b * 2048 + 64 * t);
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            c[u][j][t] = *reinterpret_cast<const u32x4_t*>(cp[j] + b * 128 + 64 * t);
        }
      }
#pragma unroll
      for (int u = 0; u < C; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[j] = product_mfma<kPeI8>(w[u][t], c[u][j][t], acc[j]);
    };
    int b = wave;
    for (; b + (kFewUnroll - 1) * kFewWaves < blocks; b += kFewUnroll * kFewWaves)
      step(b, std::integral_constant<int, kFewUnroll>{});
    for (; b < blocks; b += kFewWaves) step(b, std::integral_constant<int, 1>{});
#pragma unroll
    for (int j = 0; j < NJ; ++j) part[wave][j][lane] = acc[j];
    __syncthreads();
    // thread (j, lane): row row0 + 16 j + lane % 16, columns 16 nt + 4 (lane / 16) .. + 3
    if (wave < NJ) {
      i32x4v_t s = part[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) s += part[w][wave][lane];
      const int r = row0 + 16 * wave + (lane & 15), n = 16 * nt + 4 * (lane >> 4);
      if (r < row_end && n < p.N) {
        const float ms = p.m_scale[source_row(p, r)];
        f32x4v_t v;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const size_t col = (size_t)e * p.N + min(n + q, p.N - 1);
          v[q] = (float)s[q] * ms * p.n_scale[col];
          if (p.bias) v[q] += p.bias[col];
        }
        store_run(p, (size_t)r * p.out_ld + n, n, v);
      }
    }
    __syncthreads();  // part is read before the next tile writes it
  }
}

}  // namespace

hipError_t launch_int8_few(ProductArgs p, int rows, hipStream_t st) {
  const int bm = rows <= 16 ? 16 : 32;
  const int panels = (p.N + 15) / 16;
  const long long tiles = ((long long)(p.R / bm) + (p.E < p.R ? p.E : p.R)) * panels;
  const unsigned grid = (unsigned)((tiles < 512 ? tiles : 512) + 7) / 8 * 8;
  p.band_gm = 1;
  const dim3 g(grid), b(64 * kFewWaves);
  if (bm == 16) hipLaunchKernelGGL(int8_few_kernel<1>, g, b, 0, st, p);
  else hipLaunchKernelGGL(int8_few_kernel<2>, g, b, 0, st, p);
  return hipGetLastError();
}

}  // namespace moe
