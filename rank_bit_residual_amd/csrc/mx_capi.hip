// C ABI of the MXFP4-tensor calls (svdq_mx_*): argument validation and launches.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "mx.h"
#include "svdq_internal.h"

namespace svdq {
namespace {

constexpr int64_t kMaxMxDim = (int64_t)1 << 30;

int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return SVDQ_OK;
  if (e == hipErrorInvalidConfiguration) return set_error(SVDQ_EINVAL, std::string(what) + ": more threads than a launch holds");
  return set_error(SVDQ_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
int64_t size_of(int dtype) { return dtype == SVDQ_F32 ? 4 : 2; }

int check_mx_dtype(int dtype) {
  if (dtype != SVDQ_F32 && dtype != SVDQ_BF16 && dtype != SVDQ_F16)
    return set_error(SVDQ_EDTYPE, "dtype must be SVDQ_F32, SVDQ_BF16 or SVDQ_F16");
  return SVDQ_OK;
}

// Common start of a device call: a clean error state and a dtype these calls take.
int begin(int dtype) {
  clear_error();
  (void)hipGetLastError();  // an error that an earlier, unrelated HIP call left
  return check_mx_dtype(dtype);
}

int check_dim(int64_t v, const char* name) {
  if (v < 1 || v > kMaxMxDim) return set_error(SVDQ_EINVAL, std::string(name) + " must be in [1, 2^30]");
  return SVDQ_OK;
}

int check_tensor(const void* codes, const void* scales, const char* name) {
  if (!codes || !scales) return set_error(SVDQ_EINVAL, std::string(name) + ": NULL buffer");
  if (!aligned(codes, kAlign) || !aligned(scales, kAlign))
    return set_error(SVDQ_EINVAL, std::string(name) + ": codes and scales must be 256-byte aligned");
  return SVDQ_OK;
}

// An output pair that may be left out as a whole.
int check_out(const void* codes, const void* scales, const char* name) {
  if (!codes && !scales) return SVDQ_OK;
  return check_tensor(codes, scales, name);
}

int check_matrix(const void* p, int64_t ld, int64_t cols, int dtype, const char* name) {
  if (!p) return set_error(SVDQ_EINVAL, std::string(name) + ": NULL buffer");
  if (ld < cols) return set_error(SVDQ_EINVAL, std::string(name) + ": row stride smaller than the row");
  if (!aligned(p, size_of(dtype))) return set_error(SVDQ_EINVAL, std::string(name) + " misaligned");
  return SVDQ_OK;
}

int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need && (!ws || bytes < need || !aligned(ws, kAlign)))
    return set_error(SVDQ_EINVAL, "workspace too small or not 256-byte aligned");
  return SVDQ_OK;
}

int check_strided(const void* x, int64_t sr, int64_t sc, int dtype, const char* name) {
  if (!x) return set_error(SVDQ_EINVAL, std::string(name) + ": NULL buffer");
  if (!aligned(x, size_of(dtype))) return set_error(SVDQ_EINVAL, std::string(name) + " misaligned");
  if (sr < 0 || sc < 0) return set_error(SVDQ_EINVAL, "strides must not be negative");
  return SVDQ_OK;
}

// For calls of several launches, before the first.
int check_grid(bool fits, const char* what) {
  return fits ? SVDQ_OK : hip_status(hipErrorInvalidConfiguration, what);
}

// Row offsets inside a tile are 32-bit: 2 (kq + 1) KB.
int check_product_k(int64_t K) {
  if (K > (int64_t)1 << 27) return set_error(SVDQ_EINVAL, "products take K up to 2^27");
  return SVDQ_OK;
}

int check_act(int act) {
  if (act < SVDQ_ACT_SILU || act > SVDQ_ACT_RELU) return set_error(SVDQ_EINVAL, "unknown activation");
  return SVDQ_OK;
}

MxOut out_of(void* codes, void* scales, int64_t K) { return MxOut{(uint8_t*)codes, (uint8_t*)scales, (int)mx_kq(K)}; }

// The product's part of the four calls below: b and everything behind it.
struct Product {
  const void *b_codes, *b_scales;
  int64_t N, K;
  bool gated;
  int act, dtype;
  const void* bias;
  void* y;
  int64_t ldy;
  void* gu;
  int64_t ldgu;
};

int check_product(int64_t M, const Product& q) {
  int st;
  if ((st = check_dim(M, "M")) || (st = check_dim(q.N, q.gated ? "F" : "N")) || (q.gated && (st = check_dim(2 * q.N, "2F"))) || (st = check_dim(q.K, "K")) ||
      (st = check_product_k(q.K)) || (st = check_tensor(q.b_codes, q.b_scales, q.gated ? "w" : "b")) ||
      (st = check_matrix(q.y, q.ldy, q.N, q.dtype, q.gated ? "h" : "y")))
    return st;
  if (q.gated && (st = check_act(q.act))) return st;
  if (q.gu && (st = check_matrix(q.gu, q.ldgu, 2 * q.N, q.dtype, "gu"))) return st;
  if (q.bias && !aligned(q.bias, size_of(q.dtype))) return set_error(SVDQ_EINVAL, "bias misaligned");
  return SVDQ_OK;
}

MxGemmParams params_of(int64_t M, const Product& q, void* part) {
  MxGemmParams p{};
  p.K = q.K;
  p.b_codes = (const uint8_t*)q.b_codes;
  p.b_scales = (const uint8_t*)q.b_scales;
  p.M = (int)M;
  p.N = (int)q.N;
  p.b_rows = (int)(q.gated ? 2 * q.N : q.N);
  p.kq = (int)mx_kq(q.K);
  p.bias = q.bias;
  p.y = q.y;
  p.ldy = q.ldy;
  p.gu = q.gu;
  p.ldgu = q.ldgu;
  p.act = q.act;
  p.part = (float*)part;
  return p;
}

int product(const void* a_codes, const void* a_scales, int64_t M, const Product& q, void* workspace,
                   size_t workspace_bytes, svdq_stream_t stream) {
  int st = begin(q.dtype);
  if (st || (st = check_product(M, q)) || (st = check_tensor(a_codes, a_scales, "a"))) return st;
  const size_t need = mx_product_part_bytes(M, q.N, (int)mx_kq(q.K), q.gated);
  if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
  MxGemmParams p = params_of(M, q, workspace);
  p.a_codes = (const uint8_t*)a_codes;
  p.a_scales = (const uint8_t*)a_scales;
  return hip_status(launch_mx_product(p, q.gated, q.dtype, (hipStream_t)stream), "MXFP4 product launch");
}

// Whether the product quantises its rows itself.
bool raw_rows(int64_t M, int64_t N, int64_t K, bool gated, int64_t sc, int64_t dtype_bytes) {
  return mx_raw_rows(M, gated ? 2 * N : N, K, sc, (int)dtype_bytes) && mx_product_decodes(M, N, (int)mx_kq(K), gated);
}

// Workspace of an unquantised A: its codes and scales (unless the product quantises it), then the parts.
size_t linear_bytes(int64_t M, int64_t N, int64_t K, bool gated, int64_t sc, int64_t dtype_bytes) {
  if (raw_rows(M, N, K, gated, sc, dtype_bytes)) return 0;
  return (size_t)(mx_code_bytes(M, K) + mx_scale_bytes(M, K)) + mx_product_part_bytes(M, N, (int)mx_kq(K), gated);
}

int linear(const void* x, int64_t M, int64_t sr, int64_t sc, const Product& q, void* workspace,
                  size_t workspace_bytes, svdq_stream_t stream) {
  int st = begin(q.dtype);
  if (st || (st = check_product(M, q)) || (st = check_strided(x, sr, sc, q.dtype, "x"))) return st;
  const size_t codes = (size_t)mx_code_bytes(M, q.K), scales = (size_t)mx_scale_bytes(M, q.K);
  if ((st = check_workspace(workspace, workspace_bytes, linear_bytes(M, q.N, q.K, q.gated, sc, size_of(q.dtype))))) return st;
  uint8_t* ws = (uint8_t*)workspace;
  hipStream_t s = (hipStream_t)stream;
  if (raw_rows(M, q.N, q.K, q.gated, sc, size_of(q.dtype))) {
    MxGemmParams p = params_of(M, q, nullptr);
    p.x = x;
    p.ldx = sr;
    return hip_status(launch_mx_decode(p, q.gated, q.dtype, s), "MXFP4 product launch");
  }
  MxGemmParams p = params_of(M, q, ws + codes + scales);
  p.a_codes = ws;
  p.a_scales = ws + codes;
  MxQuantParams a{x, M, q.K, sr, sc, out_of(ws, ws + codes, q.K), MxOut{}};
  if ((st = check_grid(mx_quantize_fits(a), "mx_quantize launch")) ||
      (st = check_grid(mx_product_fits(M, q.N, (int)mx_kq(q.K), q.gated), "MXFP4 product launch")))
    return st;
  if ((st = hip_status(launch_mx_quantize(a, q.dtype, s), "mx_quantize launch"))) return st;
  return hip_status(launch_mx_product(p, q.gated, q.dtype, s), "MXFP4 product launch");
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" {

int svdq_mx_layout(int64_t rows, int64_t K, size_t* code_bytes, size_t* scale_bytes) {
  clear_error();
  int st = check_dim(rows, "rows");
  if (st || (st = check_dim(K, "K"))) return st;
  if (!code_bytes || !scale_bytes) return set_error(SVDQ_EINVAL, "NULL result pointer");
  *code_bytes = (size_t)mx_code_bytes(rows, K);
  *scale_bytes = (size_t)mx_scale_bytes(rows, K);
  return SVDQ_OK;
}

int svdq_mx_quantize(const void* x, int64_t R, int64_t C, int64_t sr, int64_t sc, int dtype, void* codes,
                     void* scales, void* codes_t, void* scales_t, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = check_dim(R, "R")) || (st = check_dim(C, "C"))) return st;
  if ((st = check_strided(x, sr, sc, dtype, "x"))) return st;
  if (!codes && !codes_t) return set_error(SVDQ_EINVAL, "nothing to quantise into");
  if ((st = check_out(codes, scales, "codes")) || (st = check_out(codes_t, scales_t, "codes_t"))) return st;
  MxQuantParams p{x, R, C, sr, sc, out_of(codes, scales, C), out_of(codes_t, scales_t, R)};
  return hip_status(launch_mx_quantize(p, dtype, (hipStream_t)stream), "mx_quantize launch");
}

int svdq_mx_dequantize(const void* codes, const void* scales, int64_t rows, int64_t K, int dtype, void* out,
                       int64_t ldo, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = check_dim(rows, "rows")) || (st = check_dim(K, "K")) || (st = check_tensor(codes, scales, "codes")) ||
      (st = check_matrix(out, ldo, K, dtype, "out")))
    return st;
  MxDequantParams p{(const uint8_t*)codes, (const uint8_t*)scales, (int)mx_kq(K), rows, K, out, ldo};
  return hip_status(launch_mx_dequantize(p, dtype, (hipStream_t)stream), "mx_dequantize launch");
}

int svdq_mx_workspace_bytes(int64_t M, int64_t N, int64_t K, int gated, size_t* bytes_out) {
  clear_error();
  int st = check_dim(M, "M");
  if (st || (st = check_dim(N, "N")) || (st = check_dim(gated ? 2 * N : N, "N")) || (st = check_dim(K, "K")) || (st = check_product_k(K))) return st;
  if (!bytes_out) return set_error(SVDQ_EINVAL, "bytes_out is NULL");
  *bytes_out = mx_product_part_bytes(M, N, (int)mx_kq(K), gated != 0);
  return SVDQ_OK;
}

int svdq_mx_product_form(int64_t M, int64_t N, int64_t K, int gated, int form[4]) {
  size_t bytes;
  const int st = svdq_mx_workspace_bytes(M, N, K, gated, &bytes);
  if (st) return st;
  if (!form) return set_error(SVDQ_EINVAL, "form is NULL");
  const MxForm f = mx_product_form(M, N, (int)mx_kq(K), gated != 0);
  form[0] = f.bm;
  form[1] = f.bn;
  form[2] = f.splits;
  form[3] = f.waves;
  return SVDQ_OK;
}

int svdq_mx_matmul(const void* a_codes, const void* a_scales, int64_t M, const void* b_codes, const void* b_scales,
                   int64_t N, int64_t K, const void* bias, int dtype, void* y, int64_t ldy, void* workspace,
                   size_t workspace_bytes, svdq_stream_t stream) {
  const Product q{b_codes, b_scales, N, K, false, 0, dtype, bias, y, ldy, nullptr, 0};
  return product(a_codes, a_scales, M, q, workspace, workspace_bytes, stream);
}

int svdq_mx_gated(const void* a_codes, const void* a_scales, int64_t M, const void* w_codes, const void* w_scales,
                  int64_t F, int64_t K, int act, int dtype, void* h, int64_t ldh, void* gu, int64_t ldgu,
                  void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  const Product q{w_codes, w_scales, F, K, true, act, dtype, nullptr, h, ldh, gu, ldgu};
  return product(a_codes, a_scales, M, q, workspace, workspace_bytes, stream);
}

int svdq_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t sc, int gated, size_t* bytes_out) {
  // the widest type is quantised inside the product least often
  return svdq_mx_linear_workspace_bytes_of(M, N, K, sc, gated, SVDQ_F32, bytes_out);
}

int svdq_mx_linear_workspace_bytes_of(int64_t M, int64_t N, int64_t K, int64_t sc, int gated, int dtype, size_t* bytes_out) {
  int st = svdq_mx_workspace_bytes(M, N, K, gated, bytes_out);
  if (st || (st = check_mx_dtype(dtype))) return st;
  if (sc < 0) return set_error(SVDQ_EINVAL, "strides must not be negative");
  *bytes_out = linear_bytes(M, N, K, gated != 0, sc, size_of(dtype));
  return SVDQ_OK;
}

int svdq_mx_linear(const void* x, int64_t M, int64_t K, int64_t sr, int64_t sc, const void* b_codes,
                   const void* b_scales, int64_t N, const void* bias, int dtype, void* y, int64_t ldy, void* workspace,
                   size_t workspace_bytes, svdq_stream_t stream) {
  const Product q{b_codes, b_scales, N, K, false, 0, dtype, bias, y, ldy, nullptr, 0};
  return linear(x, M, sr, sc, q, workspace, workspace_bytes, stream);
}

int svdq_mx_gated_linear(const void* x, int64_t M, int64_t K, int64_t sr, int64_t sc, const void* w_codes,
                         const void* w_scales, int64_t F, int act, int dtype, void* h, int64_t ldh, void* gu,
                         int64_t ldgu, void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  const Product q{w_codes, w_scales, F, K, true, act, dtype, nullptr, h, ldh, gu, ldgu};
  return linear(x, M, sr, sc, q, workspace, workspace_bytes, stream);
}

// d in both directions, then the larger of the two products' parts (they run one after the other).
static size_t backward_bytes(int64_t M, int64_t F, int64_t K, size_t at[5]) {
  size_t o = 0;
  const int64_t size[4] = {mx_code_bytes(M, 2 * F), mx_scale_bytes(M, 2 * F), mx_code_bytes(2 * F, M), mx_scale_bytes(2 * F, M)};
  for (int i = 0; i < 4; i++) {
    at[i] = o;
    o += (size_t)size[i];
  }
  at[4] = o;
  const size_t dx = mx_product_part_bytes(M, K, (int)mx_kq(2 * F), false), dw = mx_product_part_bytes(K, 2 * F, (int)mx_kq(M), false);
  return o + (dx > dw ? dx : dw);
}

int svdq_mx_gated_backward_workspace_bytes(int64_t M, int64_t F, int64_t K, size_t* bytes_out) {
  clear_error();
  int st = check_dim(M, "M");
  if (st || (st = check_dim(F, "F")) || (st = check_dim(2 * F, "2F")) || (st = check_dim(K, "K")) ||
      (st = check_product_k(2 * F)) || (st = check_product_k(M)))
    return st;
  if (!bytes_out) return set_error(SVDQ_EINVAL, "bytes_out is NULL");
  size_t at[5];
  *bytes_out = backward_bytes(M, F, K, at);
  return SVDQ_OK;
}

int svdq_mx_gated_backward(const void* dh, int64_t ldh, const void* gu, int64_t ldgu, int64_t M, int64_t F, int act,
                           int dtype, const void* w_codes, const void* w_scales, const void* x_codes, const void* x_scales,
                           int64_t K, int out_dtype, void* dx, int64_t lddx, void* dw, int64_t lddw, void* workspace,
                           size_t workspace_bytes, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = begin(out_dtype)) || (st = check_dim(F, "F")) || (st = check_act(act)) ||
      (st = check_matrix(dh, ldh, F, dtype, "dh")) || (st = check_matrix(gu, ldgu, 2 * F, dtype, "gu")))
    return st;
  Product q_dx{w_codes, w_scales, K, 2 * F, false, 0, out_dtype, nullptr, dx, lddx, nullptr, 0};
  Product q_dw{nullptr, nullptr, 2 * F, M, false, 0, out_dtype, nullptr, dw, lddw, nullptr, 0};
  size_t at[5];
  if ((st = check_product(M, q_dx)) || (st = check_dim(M, "M")) || (st = check_product_k(M)) ||
      (st = check_tensor(x_codes, x_scales, "x")) || (st = check_matrix(dw, lddw, 2 * F, out_dtype, "dw")) ||
      (st = check_workspace(workspace, workspace_bytes, backward_bytes(M, F, K, at))))
    return st;
  uint8_t* ws = (uint8_t*)workspace;
  hipStream_t s = (hipStream_t)stream;
  const MxGradParams p{dh, gu, M, F, ldh, ldgu, act, out_of(ws + at[0], ws + at[1], 2 * F), out_of(ws + at[2], ws + at[3], M)};
  if ((st = check_grid(mx_gated_grad_fits(p), "mx_gated_grad launch")) ||
      (st = check_grid(mx_product_fits(M, K, (int)mx_kq(2 * F), false), "launch of the product for dx")) ||
      (st = check_grid(mx_product_fits(K, 2 * F, (int)mx_kq(M), false), "launch of the product for dw")))
    return st;
  if ((st = hip_status(launch_mx_gated_grad(p, dtype, s), "mx_gated_grad launch"))) return st;
  MxGemmParams a = params_of(M, q_dx, ws + at[4]);
  a.a_codes = ws + at[0];
  a.a_scales = ws + at[1];
  if ((st = hip_status(launch_mx_product(a, false, out_dtype, s), "MXFP4 product launch"))) return st;
  q_dw.b_codes = ws + at[2];
  q_dw.b_scales = ws + at[3];
  MxGemmParams b = params_of(K, q_dw, ws + at[4]);
  b.a_codes = (const uint8_t*)x_codes;
  b.a_scales = (const uint8_t*)x_scales;
  return hip_status(launch_mx_product(b, false, out_dtype, s), "MXFP4 product launch");
}

int svdq_mx_gated_grad(const void* dh, int64_t ldh, const void* gu, int64_t ldgu, int64_t M, int64_t F, int act,
                       int dtype, void* codes, void* scales, void* codes_t, void* scales_t, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = check_dim(M, "M")) || (st = check_dim(F, "F")) || (st = check_dim(2 * F, "2F")) || (st = check_act(act)) ||
      (st = check_matrix(dh, ldh, F, dtype, "dh")) || (st = check_matrix(gu, ldgu, 2 * F, dtype, "gu")))
    return st;
  if (!codes && !codes_t) return set_error(SVDQ_EINVAL, "nothing to quantise into");
  if ((st = check_out(codes, scales, "codes")) || (st = check_out(codes_t, scales_t, "codes_t"))) return st;
  MxGradParams p{dh, gu, M, F, ldh, ldgu, act, out_of(codes, scales, 2 * F), out_of(codes_t, scales_t, M)};
  return hip_status(launch_mx_gated_grad(p, dtype, (hipStream_t)stream), "mx_gated_grad launch");
}

}  // extern "C"
