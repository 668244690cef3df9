// Ragged grouped products on the matrix cores: what the tile kernels of moe_product_kernels.hip
// share (operand kinds, argument block, expert lookup, fragment reads, output stores).
//
// Every product here is out[m][n] = sum_k M[m][k] N[n][k] per expert, with the n operand as the
// MFMA's A matrix and the m operand as its B matrix: a lane of a 16 x 16 MFMA then holds one output
// row m and four consecutive columns n.
//   forward   out[r][n]  : m = routed rows (K-contiguous), n = columns of W [K][N] (K-strided)
//   input grad dX[r][k'] : m = rows of dY, n = rows of W [K][N], the sum along N: both contiguous
//   weight grad dW[k'][n]: m = columns of X, n = columns of dY, the sum over the expert's rows:
//                          both strided
//   int8                 : m = code rows, n = packed weight panels, both contiguous
#pragma once

#include <type_traits>

#include "moe_internal.h"
#include "moe_tile_order.h"

namespace moe {

// element types of the tile kernels
enum ProductElt : int { kPeBf16 = 0, kPeFp16 = 1, kPeI8 = 2 };

// operand kinds: how the sum index k lies in memory
//   kOpKc   : [row][k], k contiguous, any row pitch
//   kOpKs   : [k][col], the kept index contiguous, any pitch (16-bit elements)
//   kOpPanel: int8 weights packed in panels of 16 rows x 128 k (moe_int8_pack_weights)
enum OperandKind : int { kOpKc = 0, kOpKs = 1, kOpPanel = 2 };

// output types of a product
enum ProductOut : int { kOutBf16 = 0, kOutFp16 = 1, kOutF32 = 2 };

constexpr int kProductMaxExperts = 1024;

struct ProductArgs {
  const uint8_t* n_base;   // n operand of expert 0
  size_t n_estride;        // bytes from one expert's n operand to the next (0: weight gradients)
  size_t n_pitch;          // bytes per row (kOpKc) or per k (kOpKs); kOpPanel: bytes per panel
  const uint8_t* m_base;   // m operand
  size_t m_pitch;          // bytes per row
  const int32_t* row_src;  // routed row r reads row row_src[r] / row_div (null: row r)
  int row_div;
  int src_rows;            // rows behind m_base (the bound row_src / row_div is clamped to)
  const int32_t* offsets;  // [E + 1] on the device, or null: one group of all R rows
  int E;
  int R;                   // routed rows
  int K;                   // sum length (weight gradients: unused, the expert's rows)
  int N;                   // output columns
  int M;                   // weight gradients: output rows per expert
  int split;               // weight gradients: parts the rows of an expert are split into
  void* out;
  size_t out_ld;           // elements between output rows
  int out_kind;            // ProductOut
  const float* m_scale;    // int8: per source row
  const float* n_scale;    // int8: [E][N]
  const float* bias;       // int8: [E][N] or null
  int band_gm;             // M groups per band of the tile order (big_tile_coords)
};

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4v_t __attribute__((ext_vector_type(4)));
typedef float f32x4v_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef u32x4_t u32x4_any_t __attribute__((aligned(1)));  // a 16-byte load from any address
typedef f32x4v_t f32x4_any_t __attribute__((aligned(4)));  // stores to any element
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));

template <int EL>
struct ProductTypes {
  static constexpr int kBytes = 2;
  using Acc = f32x4v_t;
};
template <>
struct ProductTypes<kPeI8> {
  static constexpr int kBytes = 1;
  using Acc = i32x4v_t;
};

// One 16 x 16 MFMA step over 64 bytes of k per row (16 of each 16 lanes): 32 elements of 16 bits, or
// 64 int8 elements summed exactly in 32-bit integers. The 16 x 16 form sums twice the k of the
// 32 x 32 form into each accumulator it touches and draws less power for it, which is what bounds
// a large product here (8192^3 bf16, both operands contiguous: 1460 TFLOP/s against 1280).
template <int EL>
__device__ __forceinline__ typename ProductTypes<EL>::Acc product_mfma(
    u32x4_t a, u32x4_t b, typename ProductTypes<EL>::Acc c) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (EL == kPeBf16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  } else if constexpr (EL == kPeFp16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a),
                                                 __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
  }
#else
  (void)a, (void)b;
  return c;
#endif
}

// ------------------------------------------------------------------------------------------------
// LDS image of one operand stage: 128 bytes of k (64 elements of 16 bits, 128 of 8) for ROWS rows.
//   contiguous kinds: row r is 128 bytes, 16-byte chunk c at slot c ^ f(r) with f(r) = r / 2 mod 8:
//     the 16 rows that a phase of a fragment read touches at one chunk lie on 16 different
//     16-byte groups of the 64 banks, and f(r + 16) = f(r), so a wave's fragments are one lane
//     address and constant offsets;
//   strided kind: k row kk is ROWS * 2 bytes, in slots of 32 bytes (16 columns), slot s at
//     s ^ g(kk). A transposing read takes, per 16 lanes, four k rows of one slot, 32 lanes k rows
//     kk .. kk + 3 and kk + 8 .. kk + 11; g spreads those eight slots over all 64 banks.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ int kc_swizzle(int row) { return (row >> 1) & 7; }

template <int ROWS>
__device__ __forceinline__ int ks_swizzle(int kk) {
  if constexpr (ROWS >= 128) return 2 * (kk & 3) + ((kk >> 3) & 1);
  else if constexpr (ROWS == 64) return (kk & 2) + ((kk >> 3) & 1);
  else return (kk >> 3) & 1;
}

// byte of 16-byte chunk `id` of a stage image (id = row * 8 + c, or kk * (ROWS / 8) + c)
template <int KIND, int ROWS>
__device__ __forceinline__ int stage_byte(int id) {
  if constexpr (KIND == kOpKs) {
    constexpr int CPR = ROWS / 8;
    const int kk = id / CPR, c = id % CPR;
    return kk * (ROWS * 2) + (((c >> 1) ^ ks_swizzle<ROWS>(kk)) << 5) + ((c & 1) << 4);
  } else {
    const int row = id >> 3, c = id & 7;
    return row * 128 + ((c ^ kc_swizzle(row)) << 4);
  }
}

// Fragment i of a wave at MFMA step t (0 or 1) of a stage: row r0 + 16 i + lane % 16, k bytes
// 64 t + 16 (lane / 16) .. + 16, r0 a multiple of the wave's rows. fragment_base is the lane's part
// of the address. The transposing read gives lane j of 16 column j of the block whose four k rows
// the 16 lanes address (lane j: row j / 4, columns 4 (j % 4) ..).
template <int KIND, int ROWS>
__device__ __forceinline__ int fragment_base(int r0, int lane) {
  if constexpr (KIND == kOpKs) {
    const int i = lane & 15;
    const int kk = 8 * (lane >> 4) + (i >> 2);
    return kk * (ROWS * 2) + (((r0 >> 4) ^ ks_swizzle<ROWS>(kk)) << 5) + ((i & 3) << 3);
  } else {
    const int row = r0 + (lane & 15);
    return row * 128 + (((lane >> 4) ^ kc_swizzle(row)) << 4);
  }
}

// the lane's place of fragment i within a stage (step 0)
template <int KIND>
__device__ __forceinline__ int fragment_place(int base, int i) {
  // (strided: slot i only touches address bits that the slot of r0 leaves zero)
  return KIND == kOpKs ? base ^ (i << 5) : base + i * 2048;
}

// fragment at `place` of the stage, step t (`off`: a constant byte offset)
template <int KIND, int ROWS>
__device__ __forceinline__ u32x4_t read_place(const uint8_t* stage, int place, int t,
                                              int off = 0) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (KIND == kOpKs) {
    const uint8_t* p0 = stage + place + t * (32 * ROWS * 2);
    const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p0);
    const s16x4_t b =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p0 + 4 * (ROWS * 2)));
    const s16x8_t v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(u32x4_t, v);
  } else {
    return *reinterpret_cast<const u32x4_t*>(stage + (place ^ (t << 6)) + off);
  }
#else
  (void)stage, (void)place, (void)t, (void)off;
  return u32x4_t{};
#endif
}

template <int KIND, int ROWS>
__device__ __forceinline__ u32x4_t read_fragment(const uint8_t* stage, int base, int i, int t) {
  if constexpr (KIND == kOpKs) return read_place<KIND, ROWS>(stage, fragment_place<KIND>(base, i), t);
  else return read_place<KIND, ROWS>(stage, base, t, i * 2048);
}

// 16 bytes at p of which the first `valid` elements (EB bytes each) exist; the rest are zero
template <int EB>
__device__ __forceinline__ u32x4_t load_chunk(const uint8_t* p, int valid) {
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (valid >= 16 / EB) {
    v = *reinterpret_cast<const u32x4_any_t*>(p);
  } else if (EB == 2 && valid > 0) {
    const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < valid) v[q >> 1] |= (uint32_t)e[q] << (16 * (q & 1));
  }
  return v;
}

// The same without a branch, for 16-bit elements of a row of at least eight, in two halves so that
// the load can be far ahead of its use: the bytes are always loaded, from the row's last eight
// elements where the chunk passes its end, from `any`, some readable 16 bytes, where it lies behind
// it; settle_chunk shifts and zeroes them.
__device__ __forceinline__ u32x4_t load_chunk_raw(const uint8_t* p, int valid,
                                                  const uint8_t* any) {
  const int miss = min(max(8 - valid, 0), 8);  // elements that do not exist
  return *reinterpret_cast<const u32x4_any_t*>(miss == 8 ? any : p - 2 * miss);
}

__device__ __forceinline__ u32x4_t settle_chunk(u32x4_t r, int valid) {
  const int miss = min(max(8 - valid, 0), 8);
  uint32_t a = r[0], b = r[1], c = r[2], d = r[3];
  if (miss & 1) {  // down by 16 bits, then by whole words; conditional moves
    a = __builtin_amdgcn_alignbit(b, a, 16);
    b = __builtin_amdgcn_alignbit(c, b, 16);
    c = __builtin_amdgcn_alignbit(d, c, 16);
    d >>= 16;
  }
  if (miss & 2) {
    a = b;
    b = c;
    c = d;
    d = 0;
  }
  if (miss & 4) {
    a = c;
    b = d;
    c = d = 0;
  }
  if (miss == 8) a = b = c = d = 0;
  return u32x4_t{a, b, c, d};
}

// ------------------------------------------------------------------------------------------------
// Expert rows and M tiles from the device-side offsets, which the host never reads. Offsets are
// clamped into [0, R] and to ascending order, so no value makes a kernel leave its buffers.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void expert_rows(const ProductArgs& p, int e, int& lo, int& hi) {
  if (!p.offsets) {
    lo = 0;
    hi = p.R;
    return;
  }
  lo = min(max(p.offsets[e], 0), p.R);
  hi = min(max(p.offsets[e + 1], lo), p.R);
}

// Rows of group g of a weight gradient: part g / E of the rows of expert g % E, parts of whole
// stages (64 rows).
__device__ __forceinline__ void wgrad_rows(const ProductArgs& p, int g, int& lo, int& hi) {
  expert_rows(p, g % p.E, lo, hi);
  if (p.split > 1) {
    const int part = ((hi - lo + p.split - 1) / p.split + 63) / 64 * 64;
    lo = min(lo + (g / p.E) * part, hi);
    hi = min(lo + part, hi);
  }
}

// The M tile table: first tile of each expert, by one scan per workgroup (the first 256 threads,
// four experts each; scratch: one int per wave). Cheaper than a launch of its own for a small call
// and invisible in a large one.
struct TileIndex {
  int first[4];  // this thread's experts: first tile of expert 4 tid + q
  int next;      // first tile after them
  int total;     // M tiles of all experts
};

template <int WAVES>
__device__ __forceinline__ TileIndex tile_index(const ProductArgs& p, int bm, int* scratch) {
  TileIndex x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int cnt[4], sum = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = 4 * tid + q;
    cnt[q] = 0;
    if (e < p.E) {
      int lo, hi;
      expert_rows(p, e, lo, hi);
      cnt[q] = (hi - lo + bm - 1) / bm;
    }
    sum += cnt[q];
  }
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) scratch[wave] = inc;
  __syncthreads();
  int base = 0;
  x.total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (w < wave) base += scratch[w];
    x.total += scratch[w];
  }
  __syncthreads();
  int f = base + inc - sum;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    x.first[q] = f;
    f += cnt[q];
  }
  x.next = f;
  return x;
}

// expert, first row and end row of M tile ti (< total), broadcast through scratch[0..2]
__device__ __forceinline__ void tile_lookup(const ProductArgs& p, const TileIndex& x, int ti,
                                            int bm, int* scratch, int& e, int& row0,
                                            int& row_end) {
  const int tid = threadIdx.x;
  if (ti >= x.first[0] && ti < x.next) {
    int q = 0;
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (ti >= x.first[i]) q = i;  // (the last expert that starts at or before ti holds it)
    int f = x.first[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (q == i) f = x.first[i];
    int lo, hi;
    expert_rows(p, 4 * tid + q, lo, hi);
    scratch[0] = 4 * tid + q;
    scratch[1] = lo + (ti - f) * bm;
    scratch[2] = hi;
  }
  __syncthreads();
  e = __builtin_amdgcn_readfirstlane(scratch[0]);
  row0 = __builtin_amdgcn_readfirstlane(scratch[1]);
  row_end = __builtin_amdgcn_readfirstlane(scratch[2]);
  __syncthreads();
}

// source row of routed row r (any index value stays inside the operand)
__device__ __forceinline__ int source_row(const ProductArgs& p, int r) {
  if (!p.row_src) return r;
  const int s = p.row_src[r] / p.row_div;
  return min(max(s, 0), p.src_rows - 1);
}

// ------------------------------------------------------------------------------------------------
// Output: four consecutive columns n .. n + 3 of row `row` (n % 4 == 0; columns from N on do not
// exist). The accumulators are float32 (or exact 32-bit integers); the only rounding is the one to
// the output type here, to nearest even by the hardware conversion, which keeps NaN and infinity.
// ------------------------------------------------------------------------------------------------
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint2 round_bf16x4(f32x4v_t v) {
  return __builtin_bit_cast(uint2, __builtin_convertvector(v, bf16x4_t));
}
__device__ __forceinline__ uint2 round_fp16x4(f32x4v_t v) {
  return __builtin_bit_cast(uint2, __builtin_convertvector(v, f16x4_t));
}

// Up to four columns n.. of a row from element `at` on. Rows of odd widths start at any element: the
// vector stores carry no alignment (a step of 1497 x 1001 x 777, three products: 59 us against 68
// with a store per element).
__device__ __forceinline__ void store_run(const ProductArgs& p, size_t at, int n, f32x4v_t v) {
  if (p.out_kind == kOutF32) {
    float* o = reinterpret_cast<float*>(p.out) + at;
    if (n + 4 <= p.N) {
      *reinterpret_cast<f32x4_any_t*>(o) = v;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < p.N) o[q] = v[q];
    }
  } else {
    const uint2 b = p.out_kind == kOutBf16 ? round_bf16x4(v) : round_fp16x4(v);
    uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + at;
    if (n + 4 <= p.N) {
      *reinterpret_cast<u32x2_any_t*>(o) = u32x2_any_t{b.x, b.y};
    } else {
      const uint16_t e[4] = {(uint16_t)b.x, (uint16_t)(b.x >> 16), (uint16_t)b.y,
                             (uint16_t)(b.y >> 16)};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < p.N) o[q] = e[q];
    }
  }
}

}  // namespace
}  // namespace moe

namespace moe {

// Host launchers (moe_product_kernels.hip); each returns hipGetLastError() after enqueueing.
hipError_t launch_grouped_gemm(ProductArgs p, int el, bool trans_w, hipStream_t st);
// ws: wgrad_split(...) > 1 parts of [E][M][N] float each
int wgrad_split(int M, int N, int E, int R);
hipError_t launch_grouped_wgrad(ProductArgs p, int el, float* ws, hipStream_t st);
hipError_t launch_int8_gemm(ProductArgs p, hipStream_t st);
// the few-row form (moe_int8_few_kernels.hip), `rows` the rows per expert on average
hipError_t launch_int8_few(ProductArgs p, int rows, hipStream_t st);

}  // namespace moe
