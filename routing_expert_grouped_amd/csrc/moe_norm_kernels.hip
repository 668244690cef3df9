// The norms before and after a block, with the block's gate and residual scale, and their
// gradients. Every reduction is float32 in a fixed order.
//
// Forward, per token: n = y r with r = (mean y^2 + eps)^(-1/2); u = a res + n w gate tau, rounded
// once; then, for the next block, z = u r' w_next from the rounded u (so the fused call gives what
// the two calls give), as 16-bit values or as int8 codes. The int8 codes are those of u w_next:
// the common factor r' only enters the scale amax r' / 127.
//
// Memory bound: each tensor is read and written once, a row staying in registers between its
// reduction and its output. Measured: post-norm with the next norm, 8192 x 6144 bf16 (403 MB) 84 us,
// 4.8 TB/s, what a copy of that size reaches; one token of 7168 about 5 us, two reductions and
// three trips to memory. Backward of both norms, 4096 x 4096 (201 MB) 44 us and 5 for the column
// sums.
#include "moe_rows.h"

namespace moe {
namespace {

template <bool FP16>
__device__ __forceinline__ void load_vec_or_one(const uint16_t* w, int c, int h, float (&f)[8]) {
  if (w) {
    unpack8<FP16>(row_load(w, c, h), f);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = 1.0f;
  }
}

template <bool FP16, int TPR, int V>
__global__ __launch_bounds__(row_block(TPR)) void norm_kernel(NormArgs a) {
  __shared__ float red[8];
  constexpr int RPB = row_block(TPR) / TPR;
  const int t = threadIdx.x % TPR;
  const int row = blockIdx.x * RPB + threadIdx.x / TPR;
  if (TPR <= 64 && row >= a.T) return;  // (whole waves; wider rows have one row per workgroup)
  const int h = a.h;
  const size_t at = (size_t)row * h;
  const float inv_h = 1.0f / (float)h;
  float u[V][8];
  u32x4_t raw[V];
#pragma unroll
  for (int v = 0; v < V; ++v) raw[v] = row_load(a.res + at, t + TPR * v, h);
#pragma unroll
  for (int v = 0; v < V; ++v) unpack8<FP16>(raw[v], u[v]);
  if (a.y) {
    float y[V][8], ss = 0.0f;
    u32x4_t yr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) yr[v] = row_load(a.y + at, t + TPR * v, h);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack8<FP16>(yr[v], y[v]);
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = __builtin_fmaf(y[v][q], y[v][q], ss);
    }
    ss = row_sum<TPR>(ss, red);
    const float r = 1.0f / sqrtf(__builtin_fmaf(ss, inv_h, a.eps));
    if (a.rstd && t == 0) a.rstd[row] = r;
    const float rt = a.tau ? r * a.tau[row] : r;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + TPR * v;
      float w[8], g[8];
      load_vec_or_one<FP16>(a.w, c, h, w);
      load_vec_or_one<FP16>(a.gate, c, h, g);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        u[v][q] = __builtin_fmaf(a.res_scale, u[v][q], y[v][q] * rt * (w[q] * g[q]));
      const u32x4_t p = pack8<FP16>(u[v]);
      row_store(a.u + at, c, h, p);
      unpack8<FP16>(p, u[v]);  // the next norm reads u as it is stored
    }
  }
  if (!a.z && !a.codes) return;
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int q = 0; q < 8; ++q) ss = __builtin_fmaf(u[v][q], u[v][q], ss);
  ss = row_sum<TPR>(ss, red);
  const float r = 1.0f / sqrtf(__builtin_fmaf(ss, inv_h, a.eps));
  if (a.rstd_next && t == 0) a.rstd_next[row] = r;
  uint32_t m = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + TPR * v;
    float w[8];
    load_vec_or_one<FP16>(a.w_next, c, h, w);
    float z[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      z[q] = u[v][q] * r * w[q];
      u[v][q] *= w[q];
      m = max(m, abs_bits(u[v][q]));
    }
    if (a.z) row_store(a.z + at, c, h, pack8<FP16>(z));
  }
  if (!a.codes) return;
  const float amax = row_max_abs<TPR>(m, red);
  const Int8Coder coder(amax);
  const int pitch = (int)int8_pitch(h);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + TPR * v;
    if (8 * c < pitch)
      *reinterpret_cast<uint2*>(a.codes + (size_t)row * pitch + 8 * c) = coder.code8(u[v]);
  }
  if (t == 0) a.scales[row] = amax * r / 127.0f;
}

// Backward, per token, with n = y r, n' = u r':
//   G  = du + r' (q - n' mean(q n')),  q = dz w_next        (the gradient of u)
//   dres = a G;   dn = G w gate tau;   dy = r (dn - n mean(dn n));   dtau = sum G n w gate
// and over the tokens: dw_next = sum dz n';  A = sum G n tau, dw = A gate, dgate = A w.
// A workgroup keeps its rows' column sums in registers (rows b, b + groups, ...) and writes them
// as one float32 partial row per sum; norm_bwd_reduce_kernel adds the partial rows in order. All of
// a row's loads go out before its first reduction, and the row stays in its 16-bit form between
// the passes over it (unpacked again in each, which costs nothing next to the loads), so the
// registers hold two column sums, the row and the three weights (rows wider than 8192 read the
// weights again for every row: they would not fit beside the rest).
template <bool FP16, int V>
struct PackedRow {
  u32x4_t v[V];
  __device__ __forceinline__ void load(const uint16_t* row, int t, int tpr, int h) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = row_load(row, t + tpr * i, h);
  }
  __device__ __forceinline__ void load_or_one(const uint16_t* row, int t, int tpr, int h) {
    if (row) {
      load(row, t, tpr, h);
    } else {
      const uint32_t one = FP16 ? 0x3c003c00u : 0x3f803f80u;
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = u32x4_t{one, one, one, one};
    }
  }
  // chunk i as float32; the empty assembly keeps an earlier unpacking from being held instead
  __device__ __forceinline__ void get(int i, float (&f)[8]) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(v[i]));
#endif
    unpack8<FP16>(v[i], f);
  }
};

template <bool FP16, int TPR, int V, bool POST, bool NEXT>
__global__ __launch_bounds__(row_block(TPR)) void norm_backward_kernel(NormBwdArgs a, int groups) {
  __shared__ float red[8];
  constexpr int RPB = row_block(TPR) / TPR;
  const int t = threadIdx.x % TPR;
  const int group = blockIdx.x * RPB + threadIdx.x / TPR;
  if (TPR <= 64 && group >= groups) return;
  const int h = a.h;
  const float inv_h = 1.0f / (float)h;
  constexpr bool HOLD = TPR <= 256;
  PackedRow<FP16, V> w, gate, wn;
  if constexpr (POST && HOLD) {
    w.load_or_one(a.w, t, TPR, h);
    gate.load_or_one(a.gate, t, TPR, h);
  }
  if constexpr (NEXT && HOLD) wn.load_or_one(a.w_next, t, TPR, h);
  float ca[V][8], cz[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int q = 0; q < 8; ++q) ca[v][q] = cz[v][q] = 0.0f;
  for (int row = group; row < a.T; row += groups) {
    const size_t at = (size_t)row * h;
    PackedRow<FP16, V> du, dz, u, y;
    if (a.du) {
      du.load(a.du + at, t, TPR, h);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) du.v[v] = u32x4_t{0u, 0u, 0u, 0u};
    }
    if constexpr (NEXT) {
      dz.load(a.dz + at, t, TPR, h);
      u.load(a.u + at, t, TPR, h);
    }
    if constexpr (POST) y.load(a.y + at, t, TPR, h);
    float g[V][8];
    if constexpr (NEXT) {
      if constexpr (!HOLD) wn.load_or_one(a.w_next, t, TPR, h);
      const float r = a.rstd_next[row];
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float n[8], q[8], wf[8];
        u.get(v, n);
        dz.get(v, q);
        wn.get(v, wf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[i] *= r;
          cz[v][i] = __builtin_fmaf(q[i], n[i], cz[v][i]);
          s = __builtin_fmaf(q[i] * wf[i], n[i], s);
        }
      }
      const float mean = row_sum<TPR>(s, red) * inv_h;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float n[8], q[8], wf[8];
        u.get(v, n);
        dz.get(v, q);
        wn.get(v, wf);
        du.get(v, g[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          g[v][i] = __builtin_fmaf(r, __builtin_fmaf(-mean, n[i] * r, q[i] * wf[i]), g[v][i]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) du.get(v, g[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = POST ? a.res_scale * g[v][q] : g[v][q];
      row_store(a.dres + at, t + TPR * v, h, pack8<FP16>(o));
    }
    if constexpr (POST) {
      if constexpr (!HOLD) {
        w.load_or_one(a.w, t, TPR, h);
        gate.load_or_one(a.gate, t, TPR, h);
      }
      const float r = a.rstd[row], tau = a.tau ? a.tau[row] : 1.0f;
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float n[8], wf[8], gf[8];
        y.get(v, n);
        w.get(v, wf);
        gate.get(v, gf);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          n[q] *= r;
          ca[v][q] = __builtin_fmaf(g[v][q] * n[q], tau, ca[v][q]);
          g[v][q] *= wf[q] * gf[q];  // dn / tau from here on
          s = __builtin_fmaf(g[v][q], n[q], s);
        }
      }
      s = row_sum<TPR>(s, red);
      if (a.dtau && t == 0) a.dtau[row] = s;
      const float mean = s * inv_h, rt = r * tau;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float n[8], o[8];
        y.get(v, n);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = rt * __builtin_fmaf(-mean, n[q] * r, g[v][q]);
        row_store(a.dy + at, t + TPR * v, h, pack8<FP16>(o));
      }
    }
  }
  // partial rows: [sum][group][h], the sums in the order A, dw_next
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + TPR * v;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int col = 8 * c + q;
      if (col >= h) continue;
      if constexpr (POST) a.partial[(size_t)group * h + col] = ca[v][q];
      if constexpr (NEXT) a.partial[((size_t)groups + group) * h + col] = cz[v][q];
    }
  }
}

// Column sums of the partial rows: 64 columns per workgroup, 16 threads per column (one wave each)
// adding every 16th partial row in order in 64 bits, then the 16 sums in order. Sixteen short
// chains of loads per column instead of one: with four, the 512 partial rows of a 4096-token batch
// took 32 us, most of it latency.
template <bool FP16>
__global__ __launch_bounds__(1024) void norm_bwd_reduce_kernel(NormBwdArgs a, int groups,
                                                               int first) {
  __shared__ double part[16][64];
  const int cx = threadIdx.x & 63, gy = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + cx;
  const bool next = blockIdx.y + first == 1;
  const float* p = a.partial + (next ? (size_t)groups * a.h : 0) + col;
  double s = 0.0;
  if (col < a.h) {
    int g = gy;
    for (; g + 7 * 16 < groups; g += 8 * 16) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = p[(size_t)(g + 16 * q) * a.h];
#pragma unroll
      for (int q = 0; q < 8; ++q) s += (double)v[q];
    }
    for (; g < groups; g += 16) s += (double)p[(size_t)g * a.h];
  }
  part[gy][cx] = s;
  __syncthreads();
  if (gy != 0 || col >= a.h) return;
  s = 0.0;
#pragma unroll
  for (int q = 0; q < 16; ++q) s += part[q][cx];
  auto vec = [&](const uint16_t* w) -> double {
    if (!w) return 1.0;
    if constexpr (FP16) return (double)(float)__builtin_bit_cast(_Float16, w[col]);
    else return (double)bf16_to_f32(w[col]);
  };
  if (next) {
    a.dw_next[col] = (float)s;
  } else {
    if (a.dw) a.dw[col] = (float)(s * vec(a.gate));
    if (a.dgate) a.dgate[col] = (float)(s * vec(a.w));
  }
}

// partial rows: one per row of a small batch, at most 512 (two workgroups per CU)
int norm_bwd_groups(int T) { return T < 512 ? T : 512; }

template <bool FP16, int TPR, int V>
void norm_backward_rows(const NormBwdArgs& a, bool post, bool next, int groups, hipStream_t st) {
  constexpr int RPB = row_block(TPR) / TPR;
  const dim3 g((groups + RPB - 1) / RPB), b(row_block(TPR));
  if (post && next)
    hipLaunchKernelGGL((norm_backward_kernel<FP16, TPR, V, true, true>), g, b, 0, st, a, groups);
  else if (post)
    hipLaunchKernelGGL((norm_backward_kernel<FP16, TPR, V, true, false>), g, b, 0, st, a, groups);
  else
    hipLaunchKernelGGL((norm_backward_kernel<FP16, TPR, V, false, true>), g, b, 0, st, a, groups);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool fp16, hipStream_t st) {
#define MOE_N(TPR, V)                                                                   \
  do {                                                                                  \
    constexpr int RPB = row_block(TPR) / TPR;                                           \
    const dim3 g((a.T + RPB - 1) / RPB), b(row_block(TPR));                             \
    if (fp16) hipLaunchKernelGGL((norm_kernel<true, TPR, V>), g, b, 0, st, a);          \
    else hipLaunchKernelGGL((norm_kernel<false, TPR, V>), g, b, 0, st, a);              \
  } while (0)
  MOE_ROW_DISPATCH(a.h, MOE_N);
#undef MOE_N
  return hipGetLastError();
}

size_t norm_bwd_partial_floats(int T, int h) { return 2 * (size_t)norm_bwd_groups(T) * h; }

hipError_t launch_norm_backward(const NormBwdArgs& a, bool post, bool next, bool fp16,
                                hipStream_t st) {
  const int groups = norm_bwd_groups(a.T);
  if (groups > 0) {
#define MOE_N(TPR, V)                                                         \
  do {                                                                        \
    if (fp16) norm_backward_rows<true, TPR, V>(a, post, next, groups, st);    \
    else norm_backward_rows<false, TPR, V>(a, post, next, groups, st);        \
  } while (0)
    MOE_ROW_DISPATCH(a.h, MOE_N);
#undef MOE_N
  }
  // one launch for the column sums that are wanted (no tokens: zeros)
  const bool want_a = post && (a.dw || a.dgate), want_z = next && a.dw_next;
  if (want_a || want_z) {
    const dim3 g((a.h + 63) / 64, want_a && want_z ? 2 : 1);
    const int first = want_a ? 0 : 1;
    if (fp16)
      hipLaunchKernelGGL((norm_bwd_reduce_kernel<true>), g, dim3(1024), 0, st, a, groups, first);
    else
      hipLaunchKernelGGL((norm_bwd_reduce_kernel<false>), g, dim3(1024), 0, st, a, groups, first);
  }
  return hipGetLastError();
}

}  // namespace moe
