// C ABI of the 8-bit tensor and layer norm calls (svdq_i8_*, svdq_layer_norm*): argument validation and launches.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "checks.h"
#include "i8.h"

namespace svdq {
namespace {

// A stage's offset in a row of tiles is 32-bit: 1024 kq.
int check_product_k(int64_t K) {
  if (K > (int64_t)1 << 26) return set_error(SVDQ_EINVAL, "products of 8-bit tensors take K up to 2^26");
  return SVDQ_OK;
}

I8Out out_of(void* codes, void* scales, int64_t K) { return I8Out{(uint8_t*)codes, (float*)scales, (int)i8_kq(K)}; }

struct Product {
  const void *b_codes, *b_scales;
  int64_t N, K;
  int dtype;
  const void* bias;
  void* y;
  int64_t ldy;
};

int check_product(int64_t M, const Product& q) {
  int st;
  if ((st = check_dim(M, "M")) || (st = check_dim(q.N, "N")) || (st = check_dim(q.K, "K")) || (st = check_product_k(q.K)) ||
      (st = check_tensor(q.b_codes, q.b_scales, "b")) || (st = check_matrix(q.y, q.ldy, q.N, q.dtype, "y")))
    return st;
  if (q.bias && !aligned(q.bias, size_of(q.dtype))) return set_error(SVDQ_EINVAL, "bias misaligned");
  return SVDQ_OK;
}

I8GemmParams params_of(int64_t M, const Product& q, void* part) {
  I8GemmParams p{};
  p.K = q.K;
  p.b_codes = (const uint8_t*)q.b_codes;
  p.b_scales = (const float*)q.b_scales;
  p.M = (int)M;
  p.N = (int)q.N;
  p.kq = (int)i8_kq(q.K);
  p.bias = q.bias;
  p.y = q.y;
  p.ldy = q.ldy;
  p.part = (int*)part;
  return p;
}

size_t round_ws(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// Whether the product quantises its rows itself.
bool raw_rows(int64_t M, int64_t N, int64_t K, int64_t sc) {
  return i8_raw_rows(M, N, K, sc) && i8_product_form(M, N, (int)i8_kq(K)).waves > 1;
}

// Workspace of an unquantised A: its codes and scales, then the scratch of quantising it and the product's parts, which take
// turns.
size_t linear_bytes(int64_t M, int64_t N, int64_t K, int64_t sr, int64_t sc) {
  if (raw_rows(M, N, K, sc)) return 0;
  const size_t part = round_ws(i8_product_part_bytes(M, N, (int)i8_kq(K))), quant = i8_quantize_bytes(M, K, sr, sc, true, false);
  return (size_t)(i8_code_bytes(M, K) + i8_scale_bytes(M)) + (part > quant ? part : quant);
}

int check_eps(double eps) {
  if (!(eps >= 0.0) || eps > 1e300) return set_error(SVDQ_EINVAL, "eps must be finite and not negative");
  return SVDQ_OK;
}

int check_params(const void* weight, const void* bias, int param_dtype, int dtype) {
  if (!weight && bias) return set_error(SVDQ_EINVAL, "a bias needs a weight");
  if (!weight) return SVDQ_OK;
  if (param_dtype != SVDQ_F32 && param_dtype != dtype)
    return set_error(SVDQ_EDTYPE, "weight and bias must be of x's dtype or SVDQ_F32");
  if (!aligned(weight, size_of(param_dtype)) || !aligned(bias, size_of(param_dtype)))
    return set_error(SVDQ_EINVAL, "weight or bias misaligned");
  return SVDQ_OK;
}

// The common part of the three forward calls.
int norm_params(NormParams& p, const void* x, int64_t ldx, int64_t M, int64_t K, const void* weight, const void* bias,
                int param_dtype, double eps, int dtype, float* mean, float* rstd) {
  int st = begin(dtype);
  if (st || (st = check_dim(M, "M")) || (st = check_dim(K, "K")) || (st = check_matrix(x, ldx, K, dtype, "x")) ||
      (st = check_params(weight, bias, param_dtype, dtype)) || (st = check_eps(eps)))
    return st;
  if (!mean != !rstd) return set_error(SVDQ_EINVAL, "mean and rstd come together");
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return set_error(SVDQ_EINVAL, "mean or rstd misaligned");
  p = NormParams{};
  p.x = x;
  p.ldx = ldx;
  p.M = M;
  p.K = K;
  p.weight = weight;
  p.bias = bias;
  p.param_f32 = param_dtype == SVDQ_F32;
  p.eps = eps;
  p.mean = mean;
  p.rstd = rstd;
  return SVDQ_OK;
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" {

int svdq_i8_layout(int64_t rows, int64_t K, size_t* code_bytes, size_t* scale_bytes) {
  clear_error();
  int st = check_dim(rows, "rows");
  if (st || (st = check_dim(K, "K"))) return st;
  if (!code_bytes || !scale_bytes) return set_error(SVDQ_EINVAL, "NULL result pointer");
  *code_bytes = (size_t)i8_code_bytes(rows, K);
  *scale_bytes = (size_t)i8_scale_bytes(rows);
  return SVDQ_OK;
}

int svdq_i8_quantize_workspace_bytes(int64_t R, int64_t C, int64_t sr, int64_t sc, int rows, int cols, size_t* bytes_out) {
  clear_error();
  int st = check_dim(R, "R");
  if (st || (st = check_dim(C, "C"))) return st;
  if (sr < 0 || sc < 0) return set_error(SVDQ_EINVAL, "strides must not be negative");
  if (!bytes_out) return set_error(SVDQ_EINVAL, "bytes_out is NULL");
  *bytes_out = i8_quantize_bytes(R, C, sr, sc, rows != 0, cols != 0);
  return SVDQ_OK;
}

int svdq_i8_quantize(const void* x, int64_t R, int64_t C, int64_t sr, int64_t sc, int dtype, void* codes, void* scales,
                     void* codes_t, void* scales_t, void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = check_dim(R, "R")) || (st = check_dim(C, "C"))) return st;
  if ((st = check_strided(x, sr, sc, dtype, "x"))) return st;
  if (!codes && !codes_t) return set_error(SVDQ_EINVAL, "nothing to quantise into");
  if ((st = check_out(codes, scales, "codes")) || (st = check_out(codes_t, scales_t, "codes_t"))) return st;
  if ((st = check_workspace(workspace, workspace_bytes, i8_quantize_bytes(R, C, sr, sc, codes != nullptr, codes_t != nullptr))) ||
      (st = check_grid(i8_quantize_fits(R, C, sr, sc, codes != nullptr, codes_t != nullptr), "i8_quantize launch")))
    return st;
  I8QuantParams p{x, R, C, sr, sc, out_of(codes, scales, C), out_of(codes_t, scales_t, R), nullptr, 0, workspace};
  return hip_status(launch_i8_quantize(p, dtype, (hipStream_t)stream), "i8_quantize launch");
}

int svdq_i8_dequantize(const void* codes, const void* scales, int64_t rows, int64_t K, int dtype, void* out, int64_t ldo,
                       svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = check_dim(rows, "rows")) || (st = check_dim(K, "K")) || (st = check_tensor(codes, scales, "codes")) ||
      (st = check_matrix(out, ldo, K, dtype, "out")))
    return st;
  I8DequantParams p{(const uint8_t*)codes, (const float*)scales, (int)i8_kq(K), rows, K, out, ldo};
  return hip_status(launch_i8_dequantize(p, dtype, (hipStream_t)stream), "i8_dequantize launch");
}

int svdq_i8_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes_out) {
  clear_error();
  int st = check_dim(M, "M");
  if (st || (st = check_dim(N, "N")) || (st = check_dim(K, "K")) || (st = check_product_k(K))) return st;
  if (!bytes_out) return set_error(SVDQ_EINVAL, "bytes_out is NULL");
  *bytes_out = i8_product_part_bytes(M, N, (int)i8_kq(K));
  return SVDQ_OK;
}

int svdq_i8_product_form(int64_t M, int64_t N, int64_t K, int form[4]) {
  size_t bytes;
  const int st = svdq_i8_workspace_bytes(M, N, K, &bytes);
  if (st) return st;
  if (!form) return set_error(SVDQ_EINVAL, "form is NULL");
  const MxForm f = i8_product_form(M, N, (int)i8_kq(K));
  form[0] = f.bm;
  form[1] = f.bn;
  form[2] = f.splits;
  form[3] = f.waves;
  return SVDQ_OK;
}

int svdq_i8_matmul(const void* a_codes, const void* a_scales, int64_t M, const void* b_codes, const void* b_scales, int64_t N,
                   int64_t K, const void* bias, int dtype, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                   svdq_stream_t stream) {
  const Product q{b_codes, b_scales, N, K, dtype, bias, y, ldy};
  int st = begin(dtype);
  if (st || (st = check_product(M, q)) || (st = check_tensor(a_codes, a_scales, "a")) ||
      (st = check_workspace(workspace, workspace_bytes, i8_product_part_bytes(M, N, (int)i8_kq(K)))))
    return st;
  I8GemmParams p = params_of(M, q, workspace);
  p.a_codes = (const uint8_t*)a_codes;
  p.a_scales = (const float*)a_scales;
  if ((st = check_grid(i8_product_fits(M, N, p.kq), "8-bit product launch"))) return st;
  return hip_status(launch_i8_product(p, dtype, (hipStream_t)stream), "8-bit product launch");
}

int svdq_i8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t sr, int64_t sc, int dtype, size_t* bytes_out) {
  int st = svdq_i8_workspace_bytes(M, N, K, bytes_out);
  if (st || (st = check_mx_dtype(dtype))) return st;
  if (sr < 0 || sc < 0) return set_error(SVDQ_EINVAL, "strides must not be negative");
  *bytes_out = linear_bytes(M, N, K, sr, sc);
  return SVDQ_OK;
}

int svdq_i8_linear(const void* x, int64_t M, int64_t K, int64_t sr, int64_t sc, const void* b_codes, const void* b_scales, int64_t N,
                   const void* bias, int dtype, void* y, int64_t ldy, void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  const Product q{b_codes, b_scales, N, K, dtype, bias, y, ldy};
  int st = begin(dtype);
  if (st || (st = check_product(M, q)) || (st = check_strided(x, sr, sc, dtype, "x")) ||
      (st = check_workspace(workspace, workspace_bytes, linear_bytes(M, N, K, sr, sc))))
    return st;
  hipStream_t s = (hipStream_t)stream;
  if ((st = check_grid(i8_product_fits(M, N, (int)i8_kq(K)), "8-bit product launch"))) return st;
  if (raw_rows(M, N, K, sc)) {
    I8GemmParams p = params_of(M, q, nullptr);
    p.x = x;
    p.ldx = sr;
    return hip_status(launch_i8_decode(p, i8_product_form(M, N, p.kq), dtype, s), "8-bit product launch");
  }
  uint8_t* ws = (uint8_t*)workspace;
  const size_t codes = (size_t)i8_code_bytes(M, K), scales = (size_t)i8_scale_bytes(M);
  I8GemmParams p = params_of(M, q, ws + codes + scales);
  p.a_codes = ws;
  p.a_scales = (const float*)(ws + codes);
  I8QuantParams a{x, M, K, sr, sc, out_of(ws, ws + codes, K), I8Out{}, nullptr, 0, ws + codes + scales};
  if ((st = check_grid(i8_quantize_fits(M, K, sr, sc, true, false), "i8_quantize launch"))) return st;
  if ((st = hip_status(launch_i8_quantize(a, dtype, s), "i8_quantize launch"))) return st;
  return hip_status(launch_i8_product(p, dtype, s), "8-bit product launch");
}

// Q(dy), Q(dy^T), then the scratch of making them and the two products' parts, which take turns.
static size_t backward_bytes(int64_t M, int64_t N, int64_t K, size_t at[5]) {
  size_t o = 0;
  const int64_t size[4] = {i8_code_bytes(M, N), i8_scale_bytes(M), i8_code_bytes(N, M), i8_scale_bytes(N)};
  for (int i = 0; i < 4; i++) {
    at[i] = o;
    o += (size_t)size[i];
  }
  at[4] = o;
  size_t most = i8_quantize_bytes(M, N, N, 1, true, true);
  for (size_t part : {i8_product_part_bytes(M, K, (int)i8_kq(N)), i8_product_part_bytes(K, N, (int)i8_kq(M))})
    if (part > most) most = part;
  return o + round_ws(most);
}

int svdq_i8_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes_out) {
  clear_error();
  int st = check_dim(M, "M");
  if (st || (st = check_dim(N, "N")) || (st = check_dim(K, "K")) || (st = check_product_k(N)) || (st = check_product_k(M)))
    return st;
  if (!bytes_out) return set_error(SVDQ_EINVAL, "bytes_out is NULL");
  size_t at[5];
  *bytes_out = backward_bytes(M, N, K, at);
  return SVDQ_OK;
}

int svdq_i8_backward_form(int64_t M, int64_t N, int64_t K, int form[2]) {
  size_t bytes;
  const int st = svdq_i8_backward_workspace_bytes(M, N, K, &bytes);
  if (st) return st;
  if (!form) return set_error(SVDQ_EINVAL, "form is NULL");
  const MxForm f = i8_pair_form(M, K, (int)i8_kq(N), K, N, (int)i8_kq(M));
  form[0] = f.bm;
  form[1] = f.bm ? f.bn : 0;
  return SVDQ_OK;
}

int svdq_i8_backward(const void* dy, int64_t lddy, int64_t M, int64_t N, int dtype, const void* w_codes, const void* w_scales,
                     const void* x_codes, const void* x_scales, int64_t K, int out_dtype, void* dx, int64_t lddx, void* dw,
                     int64_t lddw, void* db, void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = begin(out_dtype)) || (st = check_dim(M, "M")) || (st = check_dim(N, "N")) ||
      (st = check_matrix(dy, lddy, N, dtype, "dy")))
    return st;
  const Product q_dx{w_codes, w_scales, K, N, out_dtype, nullptr, dx, lddx};
  Product q_dw{nullptr, nullptr, N, M, out_dtype, nullptr, dw, lddw};
  size_t at[5];
  if ((st = check_product(M, q_dx)) || (st = check_product_k(M)) || (st = check_tensor(x_codes, x_scales, "x")) ||
      (st = check_matrix(dw, lddw, N, out_dtype, "dw")))
    return st;
  if (db && !aligned(db, size_of(out_dtype))) return set_error(SVDQ_EINVAL, "db misaligned");
  if ((st = check_workspace(workspace, workspace_bytes, backward_bytes(M, N, K, at)))) return st;
  uint8_t* ws = (uint8_t*)workspace;
  hipStream_t s = (hipStream_t)stream;
  // a column step of 1 whatever lddy: read as given, never as its transpose, so that the sums are those of dy's columns
  const I8QuantParams p{dy, M, N, lddy, 1, out_of(ws + at[0], ws + at[1], N), out_of(ws + at[2], ws + at[3], M), db, out_dtype, ws + at[4]};
  if ((st = check_grid(i8_quantize_fits(M, N, lddy, 1, true, true), "i8_quantize launch")) ||
      (st = check_grid(i8_product_fits(M, K, (int)i8_kq(N)), "launch of the product for dx")) ||
      (st = check_grid(i8_product_fits(K, N, (int)i8_kq(M)), "launch of the product for dw")))
    return st;
  if ((st = hip_status(launch_i8_quantize(p, dtype, s), "i8_quantize launch"))) return st;
  I8GemmParams a = params_of(M, q_dx, ws + at[4]);
  a.a_codes = ws + at[0];
  a.a_scales = (const float*)(ws + at[1]);
  q_dw.b_codes = ws + at[2];
  q_dw.b_scales = ws + at[3];
  I8GemmParams b = params_of(K, q_dw, ws + at[4]);
  b.a_codes = (const uint8_t*)x_codes;
  b.a_scales = (const float*)x_scales;
  return hip_status(launch_i8_products(a, b, out_dtype, s), "8-bit product launch");
}

int svdq_layer_norm(const void* x, int64_t ldx, int64_t M, int64_t K, const void* weight, const void* bias, int param_dtype,
                    double eps, int dtype, void* y, int64_t ldy, float* mean, float* rstd, svdq_stream_t stream) {
  NormParams p;
  int st = norm_params(p, x, ldx, M, K, weight, bias, param_dtype, eps, dtype, mean, rstd);
  if (st || (st = check_matrix(y, ldy, K, dtype, "y"))) return st;
  p.y = y;
  p.ldy = ldy;
  return hip_status(launch_norm(p, dtype, (hipStream_t)stream), "layer_norm launch");
}

int svdq_layer_norm_i8(const void* x, int64_t ldx, int64_t M, int64_t K, const void* weight, const void* bias, int param_dtype,
                       double eps, int dtype, void* codes, void* scales, float* mean, float* rstd, svdq_stream_t stream) {
  NormParams p;
  int st = norm_params(p, x, ldx, M, K, weight, bias, param_dtype, eps, dtype, mean, rstd);
  if (st || (st = check_tensor(codes, scales, "codes"))) return st;
  p.i8 = out_of(codes, scales, K);
  return hip_status(launch_norm(p, dtype, (hipStream_t)stream), "layer_norm launch");
}

int svdq_layer_norm_mx(const void* x, int64_t ldx, int64_t M, int64_t K, const void* weight, const void* bias, int param_dtype,
                       double eps, int dtype, void* codes, void* scales, float* mean, float* rstd, svdq_stream_t stream) {
  NormParams p;
  int st = norm_params(p, x, ldx, M, K, weight, bias, param_dtype, eps, dtype, mean, rstd);
  if (st || (st = check_tensor(codes, scales, "codes"))) return st;
  p.mx = MxOut{(uint8_t*)codes, (uint8_t*)scales, (int)mx_kq(K)};
  return hip_status(launch_norm(p, dtype, (hipStream_t)stream), "layer_norm launch");
}

int svdq_layer_norm_backward_workspace_bytes(int64_t M, int64_t K, int params, size_t* bytes_out) {
  clear_error();
  int st = check_dim(M, "M");
  if (st || (st = check_dim(K, "K"))) return st;
  if (!bytes_out) return set_error(SVDQ_EINVAL, "bytes_out is NULL");
  *bytes_out = norm_grad_bytes(M, K, params != 0);
  return SVDQ_OK;
}

int svdq_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* mean, const float* rstd, int64_t M,
                             int64_t K, const void* weight, int param_dtype, int dtype, void* dx, int64_t lddx, void* dweight,
                             void* dbias, void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = check_dim(M, "M")) || (st = check_dim(K, "K")) || (st = check_matrix(dy, lddy, K, dtype, "dy")) ||
      (st = check_matrix(x, ldx, K, dtype, "x")) || (st = check_matrix(dx, lddx, K, dtype, "dx")) ||
      (st = check_params(weight, nullptr, param_dtype, dtype)))
    return st;
  if (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)) return set_error(SVDQ_EINVAL, "mean or rstd NULL or misaligned");
  if (!weight != !dweight || !weight != !dbias) return set_error(SVDQ_EINVAL, "dweight and dbias come with a weight");
  if (weight && (!aligned(dweight, size_of(param_dtype)) || !aligned(dbias, size_of(param_dtype))))
    return set_error(SVDQ_EINVAL, "dweight or dbias misaligned");
  if ((st = check_workspace(workspace, workspace_bytes, norm_grad_bytes(M, K, weight != nullptr))) ||
      (weight && (st = check_grid(norm_grad_fits(K), "layer_norm_backward launch"))))
    return st;
  NormGradParams p{dy, x, lddy, ldx, M, K, mean, rstd, weight, param_dtype == SVDQ_F32, dx, lddx, dweight, dbias, workspace};
  return hip_status(launch_norm_grad(p, dtype, (hipStream_t)stream), "layer_norm_backward launch");
}

}  // extern "C"
