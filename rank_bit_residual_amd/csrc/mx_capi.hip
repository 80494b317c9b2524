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
  return set_error(SVDQ_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
int64_t size_of(int dtype) { return dtype == SVDQ_F32 ? 4 : 2; }

// Common start of a device call: a clean error state and a dtype these calls take.
int begin(int dtype) {
  clear_error();
  (void)hipGetLastError();  // an error that an earlier, unrelated HIP call left
  if (dtype != SVDQ_F32 && dtype != SVDQ_BF16 && dtype != SVDQ_F16)
    return set_error(SVDQ_EDTYPE, "dtype must be SVDQ_F32, SVDQ_BF16 or SVDQ_F16");
  return SVDQ_OK;
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

// The product's workspace: its float32 parts where K is split, else none.
int check_workspace(const void* ws, size_t bytes, int64_t M, int64_t N, int64_t K, bool gated) {
  const size_t need = mx_product_part_bytes(M, N, (int)mx_kq(K), gated);
  if (need && (!ws || bytes < need || !aligned(ws, kAlign)))
    return set_error(SVDQ_EINVAL, "workspace too small or not 256-byte aligned");
  return SVDQ_OK;
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
  if (!x) return set_error(SVDQ_EINVAL, "x: NULL buffer");
  if (!aligned(x, size_of(dtype))) return set_error(SVDQ_EINVAL, "x misaligned");
  if (sr < 0 || sc < 0) return set_error(SVDQ_EINVAL, "strides must not be negative");
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
  if (st || (st = check_dim(gated ? 2 * N : N, "N")) || (st = check_dim(K, "K")) || (st = check_product_k(K))) return st;
  if (!bytes_out) return set_error(SVDQ_EINVAL, "bytes_out is NULL");
  *bytes_out = mx_product_part_bytes(M, N, (int)mx_kq(K), gated != 0);
  return SVDQ_OK;
}

int svdq_mx_matmul(const void* a_codes, const void* a_scales, int64_t M, const void* b_codes, const void* b_scales,
                   int64_t N, int64_t K, const void* bias, int dtype, void* y, int64_t ldy, void* workspace,
                   size_t workspace_bytes, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = check_dim(M, "M")) || (st = check_dim(N, "N")) || (st = check_dim(K, "K")) ||
      (st = check_tensor(a_codes, a_scales, "a")) || (st = check_tensor(b_codes, b_scales, "b")) ||
      (st = check_matrix(y, ldy, N, dtype, "y")))
    return st;
  if (bias && !aligned(bias, size_of(dtype))) return set_error(SVDQ_EINVAL, "bias misaligned");
  if ((st = check_product_k(K)) || (st = check_workspace(workspace, workspace_bytes, M, N, K, false))) return st;
  MxGemmParams p{};
  p.a_codes = (const uint8_t*)a_codes;
  p.a_scales = (const uint8_t*)a_scales;
  p.b_codes = (const uint8_t*)b_codes;
  p.b_scales = (const uint8_t*)b_scales;
  p.M = (int)M;
  p.N = (int)N;
  p.b_rows = (int)N;
  p.kq = (int)mx_kq(K);
  p.bias = bias;
  p.y = y;
  p.ldy = ldy;
  p.part = (float*)workspace;
  return hip_status(launch_mx_product(p, false, dtype, (hipStream_t)stream), "mx_matmul launch");
}

int svdq_mx_gated(const void* a_codes, const void* a_scales, int64_t M, const void* w_codes, const void* w_scales,
                  int64_t F, int64_t K, int act, int dtype, void* h, int64_t ldh, void* gu, int64_t ldgu,
                  void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = check_dim(M, "M")) || (st = check_dim(2 * F, "2F")) || (st = check_dim(K, "K")) || (st = check_act(act)) ||
      (st = check_tensor(a_codes, a_scales, "a")) || (st = check_tensor(w_codes, w_scales, "w")) ||
      (st = check_matrix(h, ldh, F, dtype, "h")))
    return st;
  if (gu && (st = check_matrix(gu, ldgu, 2 * F, dtype, "gu"))) return st;
  if ((st = check_product_k(K)) || (st = check_workspace(workspace, workspace_bytes, M, F, K, true))) return st;
  MxGemmParams p{};
  p.a_codes = (const uint8_t*)a_codes;
  p.a_scales = (const uint8_t*)a_scales;
  p.b_codes = (const uint8_t*)w_codes;
  p.b_scales = (const uint8_t*)w_scales;
  p.M = (int)M;
  p.N = (int)F;
  p.b_rows = (int)(2 * F);
  p.kq = (int)mx_kq(K);
  p.y = h;
  p.ldy = ldh;
  p.gu = gu;
  p.ldgu = ldgu;
  p.act = act;
  p.part = (float*)workspace;
  return hip_status(launch_mx_product(p, true, dtype, (hipStream_t)stream), "mx_gated launch");
}

int svdq_mx_gated_grad(const void* dh, int64_t ldh, const void* gu, int64_t ldgu, int64_t M, int64_t F, int act,
                       int dtype, void* codes, void* scales, void* codes_t, void* scales_t, svdq_stream_t stream) {
  int st = begin(dtype);
  if (st || (st = check_dim(M, "M")) || (st = check_dim(2 * F, "2F")) || (st = check_act(act)) ||
      (st = check_matrix(dh, ldh, F, dtype, "dh")) || (st = check_matrix(gu, ldgu, 2 * F, dtype, "gu")))
    return st;
  if (!codes && !codes_t) return set_error(SVDQ_EINVAL, "nothing to quantise into");
  if ((st = check_out(codes, scales, "codes")) || (st = check_out(codes_t, scales_t, "codes_t"))) return st;
  MxGradParams p{dh, gu, M, F, ldh, ldgu, act, out_of(codes, scales, 2 * F), out_of(codes_t, scales_t, M)};
  return hip_status(launch_mx_gated_grad(p, dtype, (hipStream_t)stream), "mx_gated_grad launch");
}

}  // extern "C"
