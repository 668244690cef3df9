// Int8 rows and weights: per-token quantisation (optionally of silu(G) * U), and the packed weight
// layout the int8 product reads.
#include "moe_rows.h"

namespace moe {
namespace {

// One row per TPR threads: s = amax / 127, code = rint(127 v / amax). The row stays in registers
// between the maximum and the codes, so it is read once (8192 x 6144 bf16, 151 MB: 28 us, 5.4 TB/s).
// SWIGLU: the row is silu(G) * U of a [2 K] row [G | U], formed in float32 and quantised from there.
// Codes behind K, up to the pitch, are zero.
template <bool FP16, bool SWIGLU, int TPR, int V>
__global__ __launch_bounds__(row_block(TPR)) void quantize_int8_kernel(
    const uint16_t* __restrict__ x, size_t ld, int R, int K, int8_t* __restrict__ codes,
    float* __restrict__ scales) {
  __shared__ float red[8];
  constexpr int RPB = row_block(TPR) / TPR;
  const int t = threadIdx.x % TPR;
  const int row = blockIdx.x * RPB + threadIdx.x / TPR;
  if (TPR <= 64 && row >= R) return;  // (whole waves; wider rows have one row per workgroup)
  const uint16_t* xr = x + (size_t)row * ld;
  float f[V][8];
  uint32_t m = 0;
  u32x4_t raw[V], up[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    raw[v] = row_load(xr, t + TPR * v, K);
    if constexpr (SWIGLU) up[v] = row_load(xr + K, t + TPR * v, K);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    unpack8<FP16>(raw[v], f[v]);
    if constexpr (SWIGLU) {
      float g[8];
      unpack8<FP16>(up[v], g);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[v][q] = silu_f(f[v][q]) * g[q];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) m = max(m, abs_bits(f[v][q]));
  }
  const float amax = row_max_abs<TPR>(m, red);
  const Int8Coder coder(amax);
  const int pitch = (int)int8_pitch(K);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + TPR * v;
    if (8 * c < pitch)
      *reinterpret_cast<uint2*>(codes + (size_t)row * pitch + 8 * c) = coder.code8(f[v]);
  }
  if (t == 0) scales[row] = amax / 127.0f;
}

// Packed weights: [E][ceil(N / 16)][Kp / 128] blocks of 16 rows x 128 bytes, Kp = K rounded up to
// 128; rows behind N and k behind K are zero. One stage of the product reads whole blocks, and a
// 16-row fragment of a few-token product is 2 KB in a row.
__global__ __launch_bounds__(256) void int8_pack_kernel(const int8_t* __restrict__ codes, int K,
                                                        int N, size_t chunks_per_expert,
                                                        uint8_t* __restrict__ packed) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;  // 16-byte chunk of the expert
  if (i >= chunks_per_expert) return;
  const size_t e = blockIdx.y;
  const int kb = (K + 127) / 128;
  const int c = (int)(i & 7), r = (int)((i >> 3) & 15);
  const size_t blk = i >> 7;
  const int n = (int)(blk / kb) * 16 + r, k = (int)(blk % kb) * 128 + 16 * c;
  const int valid = n < N ? K - k : 0;
  const int8_t* src = codes + (e * N + n) * (size_t)K + k;
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (valid >= 16) {
    v = *reinterpret_cast<const u32x4_any_t*>(src);
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q)
      if (q < valid) v[q >> 2] |= (uint32_t)(uint8_t)src[q] << (8 * (q & 3));
  }
  *reinterpret_cast<u32x4_t*>(packed + (e * chunks_per_expert + i) * 16) = v;
}

// Weights [E][K][N] bf16 (y = x W) quantised per column: scale = amax_k / 127, packed as above. A
// workgroup takes 64 columns: one pass for the column maxima, one for the codes, transposed
// through LDS 128 k at a time.
__global__ __launch_bounds__(256) void int8_prepare_kernel(const uint16_t* __restrict__ w, int K,
                                                           int N, size_t panel_bytes,
                                                           size_t expert_bytes,
                                                           uint8_t* __restrict__ packed,
                                                           float* __restrict__ scales) {
  __shared__ uint32_t smax[4][64];
  __shared__ uint8_t tile[64][132];  // [column][k] (132: columns on different banks)
  const size_t e = blockIdx.y;
  const int n0 = blockIdx.x * 64;
  const int tid = threadIdx.x, cx = tid & 63, ky = tid >> 6;
  const int n = n0 + cx;
  const uint16_t* we = w + e * (size_t)K * N;
  uint32_t m = 0;
  if (n < N)
    for (int k = ky; k < K; k += 4) m = max(m, abs_bits(bf16_to_f32(we[(size_t)k * N + n])));
  smax[ky][cx] = m;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) m = max(m, smax[q][cx]);
  const Int8Coder coder(__uint_as_float(m));
  if (ky == 0 && n < N) scales[e * N + n] = __uint_as_float(m) / 127.0f;
  const int kb = (K + 127) / 128;
  for (int b = 0; b < kb; ++b) {
    __syncthreads();
    for (int q = ky; q < 128; q += 4) {
      const int k = 128 * b + q;
      const float v = (n < N && k < K) ? bf16_to_f32(we[(size_t)k * N + n]) : 0.0f;
      tile[cx][q] = (uint8_t)coder.code(v);
    }
    __syncthreads();
    // 64 rows x 8 chunks of 16 bytes = 512 chunks; panels behind ceil(N / 16) do not exist
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int id = u * 256 + tid, row = id >> 3, c = id & 7;
      const int panel = (n0 + row) >> 4;
      if (panel * 16 < N) {
        u32x4_t v;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[q] = *reinterpret_cast<const uint32_t*>(&tile[row][16 * c + 4 * q]);
        *reinterpret_cast<u32x4_t*>(packed + e * expert_bytes + (size_t)panel * panel_bytes +
                                    (size_t)b * 2048 + (row & 15) * 128 + 16 * c) = v;
      }
    }
  }
}

}  // namespace

hipError_t launch_quantize_int8(const uint16_t* x, size_t ld, int R, int K, bool fp16, bool swiglu,
                                int8_t* codes, float* scales, hipStream_t st) {
#define MOE_Q(TPR, V)                                                                           \
  do {                                                                                          \
    constexpr int RPB = row_block(TPR) / TPR;                                                   \
    const dim3 g((R + RPB - 1) / RPB), b(row_block(TPR));                                       \
    if (fp16 && swiglu)                                                                         \
      hipLaunchKernelGGL((quantize_int8_kernel<true, true, TPR, V>), g, b, 0, st, x, ld, R, K,  \
                         codes, scales);                                                        \
    else if (fp16)                                                                              \
      hipLaunchKernelGGL((quantize_int8_kernel<true, false, TPR, V>), g, b, 0, st, x, ld, R, K, \
                         codes, scales);                                                        \
    else if (swiglu)                                                                            \
      hipLaunchKernelGGL((quantize_int8_kernel<false, true, TPR, V>), g, b, 0, st, x, ld, R, K, \
                         codes, scales);                                                        \
    else                                                                                        \
      hipLaunchKernelGGL((quantize_int8_kernel<false, false, TPR, V>), g, b, 0, st, x, ld, R,   \
                         K, codes, scales);                                                     \
  } while (0)
  MOE_ROW_DISPATCH(K, MOE_Q);
#undef MOE_Q
  return hipGetLastError();
}

hipError_t launch_int8_pack_weights(const int8_t* codes, int E, int K, int N, uint8_t* packed,
                                    hipStream_t st) {
  const size_t chunks = (size_t)((N + 15) / 16) * ((K + 127) / 128) * 128;
  hipLaunchKernelGGL(int8_pack_kernel, dim3((unsigned)((chunks + 255) / 256), E), dim3(256), 0, st,
                     codes, K, N, chunks, packed);
  return hipGetLastError();
}

hipError_t launch_int8_prepare_weights(const uint16_t* w, int E, int K, int N, uint8_t* packed,
                                       float* scales, hipStream_t st) {
  const size_t panel = int8_pitch(K) * 16;
  hipLaunchKernelGGL(int8_prepare_kernel, dim3((N + 63) / 64, E), dim3(256), 0, st, w, K, N, panel,
                     panel * ((N + 15) / 16), packed, scales);
  return hipGetLastError();
}

}  // namespace moe
