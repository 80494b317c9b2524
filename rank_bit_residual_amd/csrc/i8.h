// 8-bit tensors with a scale for each row, and layer norm: parameter blocks and launchers of k_i8_quant.hip, k_i8_gemm.hip,
// k_i8_decode.hip and k_norm.hip (called from i8_capi.hip). Every launcher enqueues on `stream` and returns the
// hipError_t of the launch; arguments were checked by the caller.
//
// An 8-bit tensor of `rows` x K is two arrays. With kq = 2 ceil(K / 128) stages of 64 codes per row (codes past K are 0):
//   codes   int8, 1 KB tiles of 16 rows x 64 codes: row r, code k at ((r / 16) kq + k / 64) 1024 + (r % 16) 64 + k % 64,
//           rows rounded up to 16
//   scales  float32 [rows], rounded up to 64
// A tile's kilobyte is what one wave loads at once, into LDS or as operands of a 16x16x64 matrix instruction. Codes of rows
// past `rows` are neither written nor read as results. A scale that is NaN: a row that held an infinity or a NaN
// (its codes are 0).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx.h"

namespace svdq {

inline int64_t i8_kq(int64_t K) { return (K + 127) / 128 * 2; }
inline int64_t i8_code_bytes(int64_t rows, int64_t K) { return (rows + 15) / 16 * i8_kq(K) * 1024; }
inline int64_t i8_scale_bytes(int64_t rows) { return (rows + 63) / 64 * 256; }

// One 8-bit tensor to write, or codes == NULL.
struct I8Out {
  uint8_t* codes;
  float* scales;
  int kq;
};

struct I8QuantParams {
  const void* x;  // element (r, c) at r * sr + c * sc
  int64_t R, C, sr, sc;
  I8Out rows;  // R x C
  I8Out cols;  // C x R: the transpose
  void* sums;  // [C] column sums in `sums_dtype`, or NULL (with cols)
  int sums_dtype;
  void* workspace;  // i8_quantize_bytes
};

struct I8DequantParams {
  const uint8_t* codes;
  const float* scales;
  int kq;
  int64_t rows, K;
  void* out;
  int64_t ldo;
};

struct I8GemmParams {
  // unquantised A (i8_raw_rows): [M][ldx] of the output's dtype, K elements a row, or NULL
  const void* x;
  int64_t ldx, K;
  const uint8_t* a_codes;
  const float* a_scales;
  const uint8_t* b_codes;
  const float* b_scales;
  int M, N;  // output rows and columns: rows of a and of b
  int kq;
  const void* bias;  // [N] or NULL
  void* y;           // [M][ldy]
  int64_t ldy;
  int splits;  // shares of K (set by the launcher)
  int* part;   // [splits][M][N] int32 sums, i8_product_part_bytes of them
};

// Layer norm of x [M, K]: y, or the 8-bit or MXFP4 tensor of y as float32.
struct NormParams {
  const void* x;
  int64_t ldx, M, K;
  const void* weight;  // [K] or NULL
  const void* bias;    // [K] or NULL
  int param_f32;       // weight and bias are float32, else of x's dtype
  double eps;
  void* y;  // [M][ldy], or NULL
  int64_t ldy;
  I8Out i8;
  MxOut mx;
  float *mean, *rstd;  // [M], or both NULL
};

struct NormGradParams {
  const void* dy;  // [M][lddy]
  const void* x;   // [M][ldx]
  int64_t lddy, ldx, M, K;
  const float *mean, *rstd;
  const void* weight;  // [K] or NULL
  int param_f32;
  void* dx;  // [M][lddx]
  int64_t lddx;
  void *dweight, *dbias;  // [K] of the weight's dtype, or NULL
  void* workspace;        // norm_grad_bytes
};

size_t i8_quantize_bytes(int64_t R, int64_t C, int64_t sr, int64_t sc, bool rows, bool cols);
bool i8_quantize_fits(int64_t R, int64_t C, int64_t sr, int64_t sc, bool rows, bool cols);
hipError_t launch_i8_quantize(const I8QuantParams& p, int dtype, hipStream_t stream);
hipError_t launch_i8_dequantize(const I8DequantParams& p, int dtype, hipStream_t stream);

MxForm i8_product_form(int64_t M, int64_t N, int kq);
bool i8_product_fits(int64_t M, int64_t N, int kq);
size_t i8_product_part_bytes(int64_t M, int64_t N, int kq);
hipError_t launch_i8_product(const I8GemmParams& p, int dtype, hipStream_t stream);
// Two products, in one launch (in this form, unless bm is 0) or one after another, with the same results; they may share `part`.
MxForm i8_pair_form(int64_t M0, int64_t N0, int kq0, int64_t M1, int64_t N1, int kq1);
hipError_t launch_i8_products(const I8GemmParams& p, const I8GemmParams& q, int dtype, hipStream_t stream);

// The kernel for few rows: its estimated time and block shape, whether its grid fits, and whether it quantises A itself.
double i8_decode_cost(int64_t M, int64_t N, int kq, MxForm* form);
bool i8_decode_fits(int64_t M, int64_t N, const MxForm& f);
bool i8_raw_rows(int64_t M, int64_t N, int64_t K, int64_t sc);
hipError_t launch_i8_decode(const I8GemmParams& p, const MxForm& f, int dtype, hipStream_t stream);

hipError_t launch_norm(const NormParams& p, int dtype, hipStream_t stream);
size_t norm_grad_bytes(int64_t M, int64_t K, bool params);
bool norm_grad_fits(int64_t K);
hipError_t launch_norm_grad(const NormGradParams& p, int dtype, hipStream_t stream);

}  // namespace svdq
