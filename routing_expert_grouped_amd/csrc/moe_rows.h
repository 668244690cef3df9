// Rows held in registers: what the row-wise kernels (norms, int8 quantisation) share. TPR threads
// (a wave or a whole workgroup of 256 or 512) take one row of up to 8 TPR V elements; thread t
// holds the 16-byte chunks t, t + TPR, ... of the row as float32. Rows may start at any element
// address: a 16-byte access needs no alignment, and only a row's last, partial chunk is accessed
// element by element.
#pragma once

#include "moe_product.h"

namespace moe {

constexpr int kRowMax = 16384;  // widest row: 512 threads, four chunks each

namespace {

template <bool FP16>
__device__ __forceinline__ void unpack8(u32x4_t v, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (FP16) {
      typedef _Float16 h2 __attribute__((ext_vector_type(2)));
      const uint32_t w = v[q];  // (a bit cast of the element itself would read element 0)
      const h2 p = __builtin_bit_cast(h2, w);
      f[2 * q] = (float)p[0];
      f[2 * q + 1] = (float)p[1];
    } else {
      f[2 * q] = bf16_lo(v[q]);
      f[2 * q + 1] = bf16_hi(v[q]);
    }
  }
}

// eight values rounded once, to nearest even (NaN and infinity kept)
template <bool FP16>
__device__ __forceinline__ u32x4_t pack8(const float (&f)[8]) {
  const f32x4v_t a = {f[0], f[1], f[2], f[3]}, b = {f[4], f[5], f[6], f[7]};
  const uint2 x = FP16 ? round_fp16x4(a) : round_bf16x4(a);
  const uint2 y = FP16 ? round_fp16x4(b) : round_bf16x4(b);
  return u32x4_t{x.x, x.y, y.x, y.y};
}

// elements of chunk c that exist in a row of h
__device__ __forceinline__ int chunk_valid(int c, int h) { return min(max(h - 8 * c, 0), 8); }

__device__ __forceinline__ u32x4_t row_load(const uint16_t* row, int c, int h) {
  return load_chunk<2>(reinterpret_cast<const uint8_t*>(row + 8 * c), chunk_valid(c, h));
}

__device__ __forceinline__ void row_store(uint16_t* row, int c, int h, u32x4_t v) {
  const int n = chunk_valid(c, h);
  uint16_t* o = row + 8 * c;
  if (n == 8) {
    *reinterpret_cast<u32x4_any_t*>(o) = v;
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) o[q] = (uint16_t)(v[q >> 1] >> (16 * (q & 1)));
  }
}

// Sum over the TPR threads of a row, the same value in all of them: a butterfly inside each wave,
// then the waves' sums in order. `red` holds one float per wave of the workgroup; the barrier
// before the writes lets it be reused.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if constexpr (TPR > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v += red[w];
  }
  return v;
}

// Largest of the non-negative floats v, as their bit patterns: ordered like the values, with NaN
// above infinity, so a NaN in a row is not lost.
template <int TPR>
__device__ __forceinline__ float row_max_abs(uint32_t v, float* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  if constexpr (TPR > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = __uint_as_float(v);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) v = max(v, __float_as_uint(red[w]));
  }
  return __uint_as_float(v);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// int8 codes rint(127 v / amax) of a row whose largest magnitude is amax. Division by one Newton
// step on the reciprocal: q0 = a r is within a few ulps, the remainder a - q0 amax is exact in one
// fma, and adding its quotient rounds to the float32 next to the true quotient, so an exact tie
// (127 v / amax = n + 1/2, frequent: v = amax / 2) stays one and goes to even. Magnitudes near the
// ends of the float32 range are first brought to the middle by an exact power of two.
struct Int8Coder {
  float amax, rcp, pre;
  __device__ __forceinline__ explicit Int8Coder(float m) {
    pre = m < 0x1p-64f ? 0x1p64f : (m > 0x1p64f ? 0x1p-64f : 1.0f);
    amax = m * pre;
    rcp = amax > 0.0f ? __builtin_amdgcn_rcpf(amax) : 0.0f;
  }
  __device__ __forceinline__ uint32_t code(float v) const {
    const float a = v * pre * 127.0f;
    const float q0 = a * rcp;
    const float q = __builtin_fmaf(__builtin_fmaf(-q0, amax, a), rcp, q0);
    return (uint32_t)(int)__builtin_rintf(q) & 0xffu;
  }
  __device__ __forceinline__ uint2 code8(const float (&f)[8]) const {
    uint2 o;
    o.x = code(f[0]) | code(f[1]) << 8 | code(f[2]) << 16 | code(f[3]) << 24;
    o.y = code(f[4]) | code(f[5]) << 8 | code(f[6]) << 16 | code(f[7]) << 24;
    return o;
  }
};

// bytes between code rows: whole 128-byte stages of the int8 product
__host__ __device__ constexpr size_t int8_pitch(size_t K) { return (K + 127) / 128 * 128; }

}  // namespace

// Rows of width h: launch F<TPR, V> with the smallest register row that holds h.
#define MOE_ROW_DISPATCH(h, CALL)          \
  do {                                     \
    if ((h) <= 512) CALL(64, 1);           \
    else if ((h) <= 1024) CALL(64, 2);     \
    else if ((h) <= 2048) CALL(256, 1);    \
    else if ((h) <= 4096) CALL(256, 2);    \
    else if ((h) <= 6144) CALL(256, 3);    \
    else if ((h) <= 8192) CALL(256, 4);    \
    else CALL(512, 4);                     \
  } while (0)

// threads of a workgroup whose rows take TPR threads each
constexpr int row_block(int tpr) { return tpr < 256 ? 256 : tpr; }

// Host launchers (moe_int8_kernels.hip)
hipError_t launch_quantize_int8(const uint16_t* x, size_t ld, int R, int K, bool fp16, bool swiglu,
                                int8_t* codes, float* scales, hipStream_t st);
hipError_t launch_int8_pack_weights(const int8_t* codes, int E, int K, int N, uint8_t* packed,
                                    hipStream_t st);
hipError_t launch_int8_prepare_weights(const uint16_t* w, int E, int K, int N, uint8_t* packed,
                                       float* scales, hipStream_t st);

// Norms (moe_norm_kernels.hip). The forward pass: u = a res + (y r) w gate tau (or u = x where y is
// null), then optionally z = (u r') w_next, as 16-bit values or as int8 codes with a scale.
struct NormArgs {
  const uint16_t* res;      // residual stream, or the input x of a plain norm
  const uint16_t* y;        // block output, or null (no post-norm: u is res itself)
  const uint16_t* w;        // [h] or null (ones)
  const uint16_t* gate;     // [h] or null
  const float* tau;         // [T] or null
  const uint16_t* w_next;   // [h] or null (ones)
  float res_scale, eps;
  uint16_t* u;              // [T][h], post-norm only
  uint16_t* z;              // [T][h] or null
  int8_t* codes;            // [T][int8_pitch(h)] or null
  float* scales;            // [T]
  float* rstd;              // [T] or null: 1 / norm of y
  float* rstd_next;         // [T] or null: 1 / norm of u
  int T, h;
};
hipError_t launch_norm(const NormArgs& a, bool fp16, hipStream_t st);

struct NormBwdArgs {
  const uint16_t* du;       // gradient of u, or null
  const uint16_t* dz;       // gradient of z, or null
  const uint16_t* u;        // with dz
  const float* rstd_next;   // with dz
  const uint16_t* w_next;   // [h] or null
  const uint16_t* y;        // block output, or null (plain norm)
  const float* rstd;        // with y
  const uint16_t* w;        // [h] or null
  const uint16_t* gate;     // [h] or null
  const float* tau;         // [T] or null
  float res_scale;
  uint16_t* dres;           // a du_total (plain norm: du_total itself)
  uint16_t* dy;             // with y
  float* dtau;              // [T] or null
  float* dw;                // [h] or null
  float* dgate;             // [h] or null
  float* dw_next;           // [h] or null
  float* partial;           // norm_bwd_partial_floats()
  int T, h;
};
size_t norm_bwd_partial_floats(int T, int h);
// post: the norm after a block (y and its gradient); next: the norm that gave z
hipError_t launch_norm_backward(const NormBwdArgs& a, bool post, bool next, bool fp16,
                                hipStream_t st);

}  // namespace moe
