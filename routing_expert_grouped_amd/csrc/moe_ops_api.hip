// C-ABI front end of the ragged grouped products, the int8 products and the block norms: argument
// checks and launches. Nothing here allocates or synchronises; every call only enqueues kernels on
// the caller's stream.
#include "moe_rows.h"

using namespace moe;

namespace {

constexpr uintptr_t kPtrAlign = 16;
constexpr int32_t kMaxRows = 1 << 30;
constexpr int32_t kMaxWidth = 1 << 20;
// -128 * -128 * K stays below 2^31: the int8 product's 32-bit sums cannot wrap
constexpr int32_t kMaxInt8K = 131071;

bool aligned_ptr(const void* p) { return p != nullptr && ((uintptr_t)p % kPtrAlign) == 0; }
bool aligned_or_null(const void* p) { return ((uintptr_t)p % kPtrAlign) == 0; }
// a buffer of `count` elements: it may be null when it has none
bool buffer_ok(const void* p, long long count) { return count == 0 || aligned_ptr(p); }

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

bool elt_16bit(int dt) { return dt == MOE_ELT_BF16 || dt == MOE_ELT_FP16; }
bool elt_any(int dt) { return elt_16bit(dt) || dt == MOE_ELT_F32; }
int out_kind(int dt) {
  return dt == MOE_ELT_BF16 ? kOutBf16 : (dt == MOE_ELT_FP16 ? kOutFp16 : kOutF32);
}

moe_status check_gemm_shape(const moe_gemm_shape* s) {
  if (!s || s->R < 0 || s->K < 1 || s->N < 1 || s->E < 1) return MOE_EINVAL;
  if (s->E > kProductMaxExperts || s->R > kMaxRows || s->K > kMaxWidth || s->N > kMaxWidth)
    return MOE_EUNSUPPORTED;
  // tiles of 32 rows x 128 columns are counted in 32 bits
  const long long mt = (long long)s->R / 32 + s->E + 1;
  const long long w = s->K > s->N ? s->K : s->N;
  if (mt * (w / 128 + 1) > (1ll << 30)) return MOE_EUNSUPPORTED;
  // and those of a weight gradient, 64 x 64
  if ((long long)s->E * ((s->K + 63) / 64) * ((s->N + 63) / 64) > (1ll << 30))
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// gather arguments: without an index, routed row r is row r
moe_status check_gather(const int32_t* row_src, int32_t row_div, int32_t src_rows, int32_t R) {
  if (row_src) {
    if (!aligned_ptr(row_src) || row_div < 1 || src_rows < 1) return MOE_EINVAL;
  } else if (src_rows < R) {
    return MOE_EINVAL;
  }
  return MOE_OK;
}

void gather_args(ProductArgs& p, const int32_t* row_src, int32_t row_div, int32_t src_rows) {
  p.row_src = row_src;
  p.row_div = row_src ? row_div : 1;
  p.src_rows = src_rows;
}

void output_args(ProductArgs& p, void* out, size_t ld, int dt) {
  p.out = out;
  p.out_ld = ld;
  p.out_kind = out_kind(dt);
}

// out[r] = rows[src(r)] W[e]   (trans: W[e]^T), `sum` the sum's length, `cols` the output's width
moe_status grouped_product(const moe_gemm_shape* s, int dt, const void* rows, int64_t ld_rows,
                           const int32_t* row_src, int32_t row_div, int32_t src_rows,
                           const void* w, bool trans, const int32_t* offsets, void* out,
                           int64_t ld_out, int out_dt, void* stream) {
  const moe_status st = check_gemm_shape(s);
  if (st != MOE_OK) return st;
  if (!elt_16bit(dt) || (out_dt != dt && out_dt != MOE_ELT_F32)) return MOE_EINVAL;
  const int32_t sum = trans ? s->N : s->K, cols = trans ? s->K : s->N;
  if (ld_rows < sum || ld_out < cols) return MOE_EINVAL;
  const moe_status g = check_gather(row_src, row_div, src_rows, s->R);
  if (g != MOE_OK) return g;
  if (!aligned_ptr(w) || !aligned_ptr(offsets) || !buffer_ok(rows, s->R) ||
      !buffer_ok(out, s->R))
    return MOE_EINVAL;
  if (s->R == 0) return MOE_OK;
  ProductArgs p{};
  p.n_base = reinterpret_cast<const uint8_t*>(w);
  p.n_estride = (size_t)s->K * s->N * 2;
  p.n_pitch = (size_t)s->N * 2;
  p.m_base = reinterpret_cast<const uint8_t*>(rows);
  p.m_pitch = (size_t)ld_rows * 2;
  gather_args(p, row_src, row_div, src_rows);
  p.offsets = offsets;
  p.E = s->E;
  p.R = s->R;
  p.K = sum;
  p.N = cols;
  output_args(p, out, (size_t)ld_out, out_dt);
  return hip_status(launch_grouped_gemm(p, dt == MOE_ELT_FP16 ? kPeFp16 : kPeBf16, trans,
                                        as_stream(stream)));
}

moe_status check_int8_shape(const moe_gemm_shape* s) {
  const moe_status st = check_gemm_shape(s);
  if (st != MOE_OK) return st;
  return s->K > kMaxInt8K ? MOE_EUNSUPPORTED : MOE_OK;
}

size_t int8_panel_bytes(const moe_gemm_shape* s) { return int8_pitch(s->K) * 16; }
size_t int8_expert_bytes(const moe_gemm_shape* s) {
  return int8_panel_bytes(s) * (size_t)((s->N + 15) / 16);
}

moe_status int8_product(const moe_gemm_shape* s, const int8_t* codes, const float* scales,
                        const int32_t* row_src, int32_t row_div, int32_t src_rows,
                        const int32_t* offsets, const void* packed, const float* w_scales,
                        const float* bias, void* out, int64_t ld_out, int out_dt,
                        void* stream) {
  if (!elt_any(out_dt) || ld_out < s->N) return MOE_EINVAL;
  const moe_status g = check_gather(row_src, row_div, src_rows, s->R);
  if (g != MOE_OK) return g;
  if (!aligned_ptr(packed) || !aligned_ptr(w_scales) || !aligned_or_null(bias) ||
      !buffer_ok(codes, s->R) || !buffer_ok(scales, s->R) || !buffer_ok(out, s->R))
    return MOE_EINVAL;
  if (s->R == 0) return MOE_OK;
  ProductArgs p{};
  p.n_base = reinterpret_cast<const uint8_t*>(packed);
  p.n_estride = int8_expert_bytes(s);
  p.n_pitch = int8_panel_bytes(s);
  p.m_base = reinterpret_cast<const uint8_t*>(codes);
  p.m_pitch = int8_pitch(s->K);
  gather_args(p, row_src, row_div, src_rows);
  p.offsets = offsets;
  p.E = s->E;
  p.R = s->R;
  p.K = s->K;
  p.N = s->N;
  output_args(p, out, (size_t)ld_out, out_dt);
  p.m_scale = scales;
  p.n_scale = w_scales;
  p.bias = bias;
  return hip_status(launch_int8_gemm(p, as_stream(stream)));
}

moe_status check_rows(int32_t T, int32_t h, int dt) {
  if (T < 0 || h < 1 || !elt_16bit(dt)) return MOE_EINVAL;
  if (T > kMaxRows || h > kRowMax) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

const uint16_t* u16(const void* p) { return reinterpret_cast<const uint16_t*>(p); }
uint16_t* u16(void* p) { return reinterpret_cast<uint16_t*>(p); }

// eps keeps the reciprocal norm of an all-zero row finite; a NaN fails the comparison
bool eps_ok(float eps) { return eps > 0.0f && eps < 1.0f; }

}  // namespace

extern "C" {

moe_status moe_grouped_gemm(const moe_gemm_shape* s, int dt, const void* rows, int64_t ld_rows,
                            const int32_t* row_src, int32_t row_div, int32_t src_rows,
                            const void* w, const int32_t* offsets, void* out, int64_t ld_out,
                            int out_dt, void* stream) {
  return grouped_product(s, dt, rows, ld_rows, row_src, row_div, src_rows, w, false, offsets, out,
                         ld_out, out_dt, stream);
}

moe_status moe_grouped_gemm_dgrad(const moe_gemm_shape* s, int dt, const void* dy,
                                  int64_t ld_dy, const int32_t* row_src, int32_t row_div,
                                  int32_t src_rows, const void* w, const int32_t* offsets,
                                  void* dx, int64_t ld_dx, int out_dt, void* stream) {
  return grouped_product(s, dt, dy, ld_dy, row_src, row_div, src_rows, w, true, offsets, dx, ld_dx,
                         out_dt, stream);
}

size_t moe_grouped_gemm_wgrad_workspace_bytes(const moe_gemm_shape* s) {
  if (check_gemm_shape(s) != MOE_OK) return 0;
  const int split = wgrad_split(s->K, s->N, s->E, s->R);
  const size_t parts = split > 1 ? (size_t)split * s->E * s->K * s->N * sizeof(float) : 0;
  return align_up(parts + 1);
}

moe_status moe_grouped_gemm_wgrad(const moe_gemm_shape* s, int dt, const void* rows,
                                  int64_t ld_rows, const int32_t* row_src, int32_t row_div,
                                  int32_t src_rows, const void* dy, int64_t ld_dy,
                                  const int32_t* offsets, void* dw, int dw_dt, void* ws,
                                  void* stream) {
  const moe_status st = check_gemm_shape(s);
  if (st != MOE_OK) return st;
  if (!elt_16bit(dt) || (dw_dt != dt && dw_dt != MOE_ELT_F32)) return MOE_EINVAL;
  if (ld_rows < s->K || ld_dy < s->N) return MOE_EINVAL;
  const moe_status g = check_gather(row_src, row_div, src_rows, s->R);
  if (g != MOE_OK) return g;
  if (!aligned_ptr(dw) || !aligned_ptr(offsets) || !aligned_ptr(ws) || !buffer_ok(rows, s->R) ||
      !buffer_ok(dy, s->R))
    return MOE_EINVAL;
  ProductArgs p{};
  p.n_base = reinterpret_cast<const uint8_t*>(dy);
  p.n_pitch = (size_t)ld_dy * 2;
  p.m_base = reinterpret_cast<const uint8_t*>(rows);
  p.m_pitch = (size_t)ld_rows * 2;
  gather_args(p, row_src, row_div, src_rows);
  p.offsets = offsets;
  p.E = s->E;
  p.R = s->R;
  p.N = s->N;
  p.M = s->K;
  output_args(p, dw, (size_t)s->N, dw_dt);
  return hip_status(launch_grouped_wgrad(p, dt == MOE_ELT_FP16 ? kPeFp16 : kPeBf16,
                                         reinterpret_cast<float*>(ws), as_stream(stream)));
}

size_t moe_int8_pitch(int32_t K) { return K < 1 ? 0 : int8_pitch(K); }

moe_status moe_quantize_int8(int32_t R, int32_t K, int dt, const void* x, int64_t ld_x,
                             int swiglu, int8_t* codes, float* scales, void* stream) {
  const moe_status st = check_rows(R, K, dt);
  if (st != MOE_OK) return st;
  if ((swiglu != 0 && swiglu != 1) || ld_x < (int64_t)K * (swiglu ? 2 : 1)) return MOE_EINVAL;
  if (!buffer_ok(x, R) || !buffer_ok(codes, R) || !buffer_ok(scales, R)) return MOE_EINVAL;
  if (R == 0) return MOE_OK;
  return hip_status(launch_quantize_int8(u16(x), (size_t)ld_x, R, K, dt == MOE_ELT_FP16,
                                         swiglu != 0, codes, scales, as_stream(stream)));
}

size_t moe_int8_weight_bytes(const moe_gemm_shape* s) {
  return check_int8_shape(s) == MOE_OK ? int8_expert_bytes(s) * (size_t)s->E : 0;
}

moe_status moe_int8_pack_weights(const moe_gemm_shape* s, const int8_t* w_codes, void* packed,
                                 void* stream) {
  const moe_status st = check_int8_shape(s);
  if (st != MOE_OK) return st;
  if (!aligned_ptr(w_codes) || !aligned_ptr(packed)) return MOE_EINVAL;
  return hip_status(launch_int8_pack_weights(w_codes, s->E, s->K, s->N,
                                             reinterpret_cast<uint8_t*>(packed),
                                             as_stream(stream)));
}

moe_status moe_int8_prepare_weights(const moe_gemm_shape* s, const uint16_t* w, void* packed,
                                    float* w_scales, void* stream) {
  const moe_status st = check_int8_shape(s);
  if (st != MOE_OK) return st;
  if (!aligned_ptr(w) || !aligned_ptr(packed) || !aligned_ptr(w_scales)) return MOE_EINVAL;
  return hip_status(launch_int8_prepare_weights(w, s->E, s->K, s->N,
                                                reinterpret_cast<uint8_t*>(packed), w_scales,
                                                as_stream(stream)));
}

moe_status moe_gemm_int8(const moe_gemm_shape* s, const int8_t* codes, const float* scales,
                         const void* packed, const float* w_scales, const float* bias, void* out,
                         int64_t ld_out, int out_dt, void* stream) {
  const moe_status st = check_int8_shape(s);
  if (st != MOE_OK) return st;
  if (s->E != 1) return MOE_EINVAL;
  return int8_product(s, codes, scales, nullptr, 1, s->R, nullptr, packed, w_scales, bias, out,
                      ld_out, out_dt, stream);
}

moe_status moe_grouped_gemm_int8(const moe_gemm_shape* s, const int8_t* codes, const float* scales,
                                 const int32_t* row_src, int32_t row_div, int32_t src_rows,
                                 const int32_t* offsets, const void* packed, const float* w_scales,
                                 const float* bias, void* out, int64_t ld_out, int out_dt,
                                 void* stream) {
  const moe_status st = check_int8_shape(s);
  if (st != MOE_OK) return st;
  if (!aligned_ptr(offsets)) return MOE_EINVAL;
  return int8_product(s, codes, scales, row_src, row_div, src_rows, offsets, packed, w_scales,
                      bias, out, ld_out, out_dt, stream);
}

moe_status moe_pre_norm(int32_t T, int32_t h, int dt, const void* x, const void* w, float eps,
                        void* z, int8_t* codes, float* scales, float* rstd, void* stream) {
  const moe_status st = check_rows(T, h, dt);
  if (st != MOE_OK) return st;
  if (!eps_ok(eps)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!aligned_ptr(x) || !aligned_or_null(w) || !aligned_or_null(z) || !aligned_or_null(codes) ||
      !aligned_or_null(scales) || !aligned_or_null(rstd))
    return MOE_EINVAL;
  if ((!z && !codes) || (codes != nullptr) != (scales != nullptr)) return MOE_EINVAL;
  NormArgs a{};
  a.res = u16(x);
  a.w_next = u16(w);
  a.eps = eps;
  a.z = u16(z);
  a.codes = codes;
  a.scales = scales;
  a.rstd_next = rstd;
  a.T = T;
  a.h = h;
  return hip_status(launch_norm(a, dt == MOE_ELT_FP16, as_stream(stream)));
}

moe_status moe_post_norm(int32_t T, int32_t h, int dt, const void* res, const void* y,
                         const void* w, const void* gate, const float* token_gate, float res_scale,
                         float eps, void* u, float* rstd, const void* w_next, void* z,
                         int8_t* codes, float* scales, float* rstd_next, void* stream) {
  const moe_status st = check_rows(T, h, dt);
  if (st != MOE_OK) return st;
  if (!eps_ok(eps)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!aligned_ptr(res) || !aligned_ptr(y) || !aligned_ptr(u) || !aligned_or_null(w) ||
      !aligned_or_null(gate) || !aligned_or_null(token_gate) || !aligned_or_null(rstd) ||
      !aligned_or_null(w_next) || !aligned_or_null(z) || !aligned_or_null(codes) ||
      !aligned_or_null(scales) || !aligned_or_null(rstd_next))
    return MOE_EINVAL;
  if ((codes != nullptr) != (scales != nullptr)) return MOE_EINVAL;
  if (!z && !codes && (w_next || rstd_next)) return MOE_EINVAL;
  NormArgs a{};
  a.res = u16(res);
  a.y = u16(y);
  a.w = u16(w);
  a.gate = u16(gate);
  a.tau = token_gate;
  a.res_scale = res_scale;
  a.eps = eps;
  a.u = u16(u);
  a.rstd = rstd;
  a.w_next = u16(w_next);
  a.z = u16(z);
  a.codes = codes;
  a.scales = scales;
  a.rstd_next = rstd_next;
  a.T = T;
  a.h = h;
  return hip_status(launch_norm(a, dt == MOE_ELT_FP16, as_stream(stream)));
}

size_t moe_norm_backward_workspace_bytes(int32_t T, int32_t h) {
  if (check_rows(T, h, MOE_ELT_BF16) != MOE_OK) return 0;
  return align_up(norm_bwd_partial_floats(T, h) * sizeof(float) + 1);
}

moe_status moe_pre_norm_backward(int32_t T, int32_t h, int dt, const void* dz, const void* x,
                                 const float* rstd, const void* w, const void* d_res, void* dx,
                                 float* dw, void* ws, void* stream) {
  const moe_status st = check_rows(T, h, dt);
  if (st != MOE_OK) return st;
  if (!buffer_ok(dz, T) || !buffer_ok(x, T) || !buffer_ok(rstd, T) || !buffer_ok(dx, T) ||
      !aligned_or_null(w) || !aligned_or_null(d_res) || !aligned_or_null(dw) || !aligned_ptr(ws))
    return MOE_EINVAL;
  NormBwdArgs a{};
  a.du = u16(d_res);
  a.dz = u16(dz);
  a.u = u16(x);
  a.rstd_next = rstd;
  a.w_next = u16(w);
  a.dres = u16(dx);
  a.dw_next = dw;
  a.partial = reinterpret_cast<float*>(ws);
  a.T = T;
  a.h = h;
  return hip_status(launch_norm_backward(a, false, true, dt == MOE_ELT_FP16, as_stream(stream)));
}

moe_status moe_post_norm_backward(int32_t T, int32_t h, int dt, const void* du, const void* y,
                                  const float* rstd, const void* w, const void* gate,
                                  const float* token_gate, float res_scale, const void* dz,
                                  const void* u, const float* rstd_next, const void* w_next,
                                  void* dres, void* dy, float* dw, float* dgate,
                                  float* dtoken_gate, float* dw_next, void* ws, void* stream) {
  const moe_status st = check_rows(T, h, dt);
  if (st != MOE_OK) return st;
  if (!buffer_ok(y, T) || !buffer_ok(rstd, T) || !buffer_ok(dres, T) || !buffer_ok(dy, T) ||
      !aligned_or_null(du) || !aligned_or_null(w) || !aligned_or_null(gate) ||
      !aligned_or_null(token_gate) || !aligned_or_null(dz) || !aligned_or_null(u) ||
      !aligned_or_null(rstd_next) || !aligned_or_null(w_next) || !aligned_or_null(dw) ||
      !aligned_or_null(dgate) || !aligned_or_null(dtoken_gate) || !aligned_or_null(dw_next) ||
      !aligned_ptr(ws))
    return MOE_EINVAL;
  // the next norm's gradient comes with what its forward read and kept; one of du, dz is given
  const bool next = dz != nullptr || (T == 0 && dw_next);
  if (T > 0 && next && (!u || !rstd_next)) return MOE_EINVAL;
  if (T > 0 && !du && !dz) return MOE_EINVAL;
  if (!next && (u || rstd_next || w_next || dw_next)) return MOE_EINVAL;
  NormBwdArgs a{};
  a.du = u16(du);
  a.dz = u16(dz);
  a.u = u16(u);
  a.rstd_next = rstd_next;
  a.w_next = u16(w_next);
  a.y = u16(y);
  a.rstd = rstd;
  a.w = u16(w);
  a.gate = u16(gate);
  a.tau = token_gate;
  a.res_scale = res_scale;
  a.dres = u16(dres);
  a.dy = u16(dy);
  a.dtau = dtoken_gate;
  a.dw = dw;
  a.dgate = dgate;
  a.dw_next = dw_next;
  a.partial = reinterpret_cast<float*>(ws);
  a.T = T;
  a.h = h;
  return hip_status(launch_norm_backward(a, true, next, dt == MOE_ELT_FP16, as_stream(stream)));
}

}  // extern "C"
