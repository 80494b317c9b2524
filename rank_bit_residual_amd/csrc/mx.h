// MXFP4 tensors made on the device: parameter blocks and launchers of k_mx_quant.hip and
// k_mx_gemm.hip (called from mx_capi.hip). Every launcher enqueues on `stream` and returns the
// hipError_t of the launch; arguments were checked by the caller.
//
// An MXFP4 tensor of `rows` x K (blocks of 32 along K) is two arrays. With kq = 2 ceil(K / 256)
// stages of 128 codes per row (codes past K are 0, their blocks' scale byte 0):
//   codes   1 KB tiles of 16 rows x 128 codes (mx_code_tile_offset), rows rounded up to 16
//   scales  E8M0 bytes, 256-byte tiles of 64 rows x 4 blocks (mx_scale_tiled_index), rows
//           rounded up to 64
// Both are the layouts of the prepared MXFP4 weights. Rows past `rows` are neither written nor
// read. A scale byte of 255 is NaN: a block that held an infinity or a NaN (its codes are 0).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace svdq {

inline int64_t mx_kq(int64_t K) { return (K + 255) / 256 * 2; }
inline int64_t mx_code_bytes(int64_t rows, int64_t K) { return (rows + 15) / 16 * mx_kq(K) * 1024; }
inline int64_t mx_scale_bytes(int64_t rows, int64_t K) { return (rows + 63) / 64 * mx_kq(K) * 256; }

// One MXFP4 tensor to write, or codes == NULL.
struct MxOut {
  uint8_t* codes;
  uint8_t* scales;
  int kq;
};

struct MxQuantParams {
  const void* x;  // element (r, c) at r * sr + c * sc
  int64_t R, C, sr, sc;
  MxOut rows;  // R x C
  MxOut cols;  // C x R: the transpose
};

struct MxDequantParams {
  const uint8_t* codes;
  const uint8_t* scales;
  int kq;
  int64_t rows, K;
  void* out;
  int64_t ldo;
};

// Whether the decode kernel quantises A itself: always for one row; for a few, where doing it again in every block is
// shorter than a launch of its own (1.9 us). A block's share costs 0.035 us (M + 4) for each 128-code stage of a wave in 16-bit
// types, twice that in float32. Measured as one launch against two (quantise, product), us on the GPU's clock:
//   16-bit   K = 2048, 16 rows x 1024 columns 4.2 and 4.8; K = 4096, 8 rows 5.6 and 5.6, 16 rows 6.8 and 5.7; K = 8192, 2 rows 6.6 and
//            6.4, 16 rows 11.3 and 6.9; K = 65536, 16 rows 77 and 27
//   float32  K = 1024, 16 rows 4.0 and 4.6; K = 2048, 8 rows 4.7 and 4.7; K = 4096, 4 rows 6.3 and 5.5, 16 rows 11.2 and 5.7
// Past 4096 rows of b a part of it hides behind the reading of b (16-bit, 4 rows x 8192: K = 8192 10.0 and 11.0, K = 16384 17.4 and 16.8),
// up to 32768 rows of a times b, where the second reading of x counts.
inline bool mx_raw_rows(int64_t M, int64_t b_rows, int64_t K, int64_t sc, int dtype_bytes) {
  if (sc != 1 || M == 1) return sc == 1;
  const int64_t most = dtype_bytes == 2 && b_rows > 4096 ? 200000 : 110000;
  return M <= 16 && M * b_rows <= 32768 && (M + 4) * K * dtype_bytes <= most;
}
struct MxGemmParams {
  // unquantised A (mx_raw_rows): [M][ldx] of the output's dtype, K elements a row, or NULL
  const void* x;
  int64_t ldx, K;
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const uint8_t* b_codes;
  const uint8_t* b_scales;
  int M, N;    // output rows and columns
  int b_rows;  // rows of b: N, or 2 N for the gated product (gate rows, then up rows)
  int kq;
  const void* bias;  // [N] or NULL
  void* y;           // [M][ldy]
  int64_t ldy;
  void* gu;  // gated: [M][ldgu] pre-activations (gate, then up), or NULL
  int64_t ldgu;
  int act;
  int splits;   // shares of K (set by the launcher)
  float* part;  // [splits][M][b_rows] float32 sums, mx_product_part_bytes of them
};

struct MxGradParams {
  const void* dh;  // [M][ldh]
  const void* gu;  // [M][ldgu]: gate pre-activations, then up
  int64_t M, F, ldh, ldgu;
  int act;
  MxOut rows;  // M x 2F: [dg | du]
  MxOut cols;  // 2F x M: the transpose
};

// A launch holds fewer than 2^32 threads along a dimension of its grid; a launcher refuses more
// (hipErrorInvalidConfiguration). A call of several launches asks mx_*_fits of each before the first, so that a refused call
// has run nothing.
inline bool mx_fits_grid(int64_t blocks, int threads) { return blocks < (int64_t)0x100000000 / threads; }

bool mx_quantize_fits(const MxQuantParams& p);
bool mx_gated_grad_fits(const MxGradParams& p);
bool mx_product_fits(int64_t M, int64_t N, int kq, bool gated);
hipError_t launch_mx_quantize(const MxQuantParams& p, int dtype, hipStream_t stream);
hipError_t launch_mx_dequantize(const MxDequantParams& p, int dtype, hipStream_t stream);
hipError_t launch_mx_gated_grad(const MxGradParams& p, int dtype, hipStream_t stream);
// How a product is cut: output tiles of bm x bn (rows of a by rows of b: a gated tile holds half gate rows, half up rows),
// K in `splits` shares over blocks, which a second kernel joins, and in `waves` shares over the waves of a block, which are
// joined in LDS (1: the tile kernels).
struct MxForm {
  int bm, bn, splits, waves;
};
MxForm mx_product_form(int64_t M, int64_t N, int kq, bool gated);
// The block shape of the kernel for few rows, and whether its grid fits.
MxForm mx_decode_form(int64_t M, int64_t N, int kq, bool gated);
bool mx_decode_fits(int64_t M, int64_t N, int kq, bool gated);
// Whether the product's launch is that kernel (the only one that takes an unquantised A).
bool mx_product_decodes(int64_t M, int64_t N, int kq, bool gated);
// Bytes of float32 parts that the product's launch writes and reads (0: K is not split).
size_t mx_product_part_bytes(int64_t M, int64_t N, int kq, bool gated);
hipError_t launch_mx_decode(const MxGemmParams& p, bool gated, int dtype, hipStream_t stream);
hipError_t launch_mx_product(const MxGemmParams& p, bool gated, int dtype, hipStream_t stream);

}  // namespace svdq
