// Elementwise kernels on 8-bit tensors for gfx950:
//   * k_i8_rows        Q(x) of each row: its largest magnitude, its scale, its codes;
//   * k_i8_colmax, k_i8_colscale, k_i8_cols   the same of each column, as a tensor of the transpose;
//   * k_i8_dequantize  the values of a tensor.
//
// s = float32(max|x| / 127), and a code is the nearest integer to x / s, ties to even, decided exactly (code8, mend8).
//
// A row is read once: it stays in the registers of the threads that share it while they agree on its maximum. A column's maximum
// comes before its first code, so columns are read twice: partial maxima (and sums) of strips of rows, their join, then the codes,
// which change places through LDS as bytes. All kernels are bound by memory; 8192 x 12288 bf16: rows 62 us (4.8 TB/s), columns 97, both 139
// in captured calls (by trace of eager ones 92 for rows and maxima, 5 for the join and 55 for the columns' codes), the values of a tensor 54
// (5.6 TB/s).
#include <type_traits>

#include "i8.h"
#include "i8_device.h"

namespace svdq {
namespace dev {

// Elements [c, c + 8) of a row of C elements with step sc, zeros past its end.
template <class DT>
__device__ inline Vec8<DT> load8_step(const typename DT::T* row, int64_t c, int64_t C, int64_t sc) {
  if (sc == 1) return load8<DT>(row, c, C);
  Vec8<DT> v = zero8<DT>();
#pragma unroll
  for (int q = 0; q < 8; q++) {
    if (c + q >= C) continue;
    const typename DT::T e = row[(c + q) * sc];
    if constexpr (DT::size == 4)
      v.w[q] = __float_as_uint(e);
    else
      v.w[q >> 1] |= (u32)e << (16 * (q & 1));
  }
  return v;
}

template <class DT>
__device__ inline void store_codes8(const I8Out& o, int64_t row, int64_t c, const Vec8<DT>& v, const Scale8& q) {
  float e[8];
#pragma unroll
  for (int k = 0; k < 8; k++) e[k] = elem<DT>(v, k);
  *reinterpret_cast<v2u*>(o.codes + i8_at(row, c, o.kq)) = codes8x8(e, q);
}

// ------------------------------------------------------------------------------ rows
// Largest magnitudes of eight columns: pairs of bits in 16-bit types.
template <class DT>
struct Most8 {
  u32 w[DT::size * 2];
};
template <class DT>
__device__ inline void add_most(Most8<DT>& m, const Vec8<DT>& v) {
#pragma unroll
  for (int k = 0; k < DT::size * 2; k++) {
    if constexpr (DT::size == 4)
      m.w[k] = max(m.w[k], v.w[k] & 0x7FFFFFFFu);
    else
      m.w[k] = max_pairs(m.w[k], v.w[k] & 0x7FFF7FFFu);
  }
}
template <class DT>
__device__ inline u32 most_at(const Most8<DT>& m, int k) {
  if constexpr (DT::size == 4)
    return m.w[k];
  else
    return __float_as_uint(DT::load((uint16_t)(m.w[k >> 1] >> (16 * (k & 1)))));
}

// T threads share a row of contiguous elements, eight at least, and hold NV times eight each; NV = 0: the row is read twice instead,
// whatever its length and step. A
// block takes rows one after another, the next on its way while one is worked on. COLS: its threads keep the maxima of their columns too
// (and SUMS, their sums), over all the rows that the block takes, and leave them in row blockIdx.x of `part` (`sums`).
enum { ROWS_ALONE, ROWS_AND_MAXIMA, ROWS_MAXIMA_AND_SUMS };
template <class DT, int T, int NV, int COLS>
__global__ __launch_bounds__(T < 256 ? 256 : T, COLS ? 4 : 1) void k_i8_rows(I8QuantParams p, u32* part, float* sums) {
  typedef typename DT::T E;
  constexpr int RPB = T < 256 ? 256 / T : 1, WAVES = T / 64, N = NV ? NV : 1;
  static_assert(COLS == ROWS_ALONE || (NV && RPB == 1), "a block's threads own their columns");
  __shared__ u32 red[2][RPB][4 * WAVES];
  const int t = threadIdx.x % T, sub = threadIdx.x / T;
  const int64_t Kp = (int64_t)p.rows.kq * 64, step = (int64_t)gridDim.x * RPB;
  auto at = [&](int j) { return (int64_t)(j * T + t) * 8; };
  auto load = [&](Vec8<DT>(&v)[N], int64_t row) {
    const E* x = reinterpret_cast<const E*>(p.x) + row * p.sr;
#pragma unroll
    for (int j = 0; j < NV; j++) {
      v[j] = load8_last<DT>(x, at(j), p.C);
    }
  };
  // the threads of a block stay together (they share barriers): past the last row some repeat it
  int64_t first = (int64_t)blockIdx.x * RPB;
  Vec8<DT> v[N], next[N];
  load(v, min(first + sub, p.R - 1));
  Most8<DT> cmax[COLS ? N : 1] = {};
  float csum[COLS == ROWS_MAXIMA_AND_SUMS ? N : 1][8] = {};
  int flip = 0;
  for (; first < p.R; first += step, flip ^= 1) {
    const int64_t row = min(first + sub, p.R - 1);
    if (first + step < p.R) load(next, min(first + step + sub, p.R - 1));
    const E* x = reinterpret_cast<const E*>(p.x) + row * p.sr;
    u32 most = 0;
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; j++) {
        fit8<DT>(v[j], at(j), p.C);
        most = max(most, amax_bits<DT>(v[j].w));
      }
    } else {
      for (int64_t c = (int64_t)t * 8; c < p.C; c += T * 8) {
        v[0] = load8_step<DT>(x, c, p.C, p.sc);
        most = max(most, amax_bits<DT>(v[0].w));
      }
    }
    if constexpr (WAVES > 1) {
      most = row_join(most, umax2);
      // two buffers: a wave may reach the next row's write while others still read this one's
      if ((t & 15) == 0) red[flip][sub][t >> 4] = most;
      lds_barrier();
      most = waves_join<WAVES>(red[flip][sub], umax2);
    } else {
      most = wave_umax(most);
    }
    const Scale8 q = scale8(most);
    if (t == 0) p.rows.scales[row] = q.s;
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; j++) {
        if (at(j) < Kp) store_codes8<DT>(p.rows, row, at(j), v[j], q);
        if constexpr (COLS != ROWS_ALONE) add_most<DT>(cmax[j], v[j]);
        if constexpr (COLS == ROWS_MAXIMA_AND_SUMS) {
#pragma unroll
          for (int k = 0; k < 8; k++) csum[j][k] += elem<DT>(v[j], k);
        }
        v[j] = next[j];
      }
    } else {
      for (int64_t c = (int64_t)t * 8; c < Kp; c += T * 8) store_codes8<DT>(p.rows, row, c, load8_step<DT>(x, c, p.C, p.sc), q);
    }
  }
  if constexpr (COLS != ROWS_ALONE) {
#pragma unroll
    for (int j = 0; j < NV; j++) {
      if (at(j) >= p.C) continue;
      float m[8];
#pragma unroll
      for (int k = 0; k < 8; k++) m[k] = __uint_as_float(most_at<DT>(cmax[j], k));
      store8<MxF32>(reinterpret_cast<float*>(part) + blockIdx.x * p.C, at(j), p.C, m);
      if constexpr (COLS == ROWS_MAXIMA_AND_SUMS) store8<MxF32>(sums + blockIdx.x * p.C, at(j), p.C, csum[j]);
    }
  }
}

// ------------------------------------------------------------------------------ columns
// Partial maxima (bits of float32) and, SUMS, sums of strip `blockIdx.y` of rows: 512 columns a block, a wave a row.
template <class DT, bool SUMS>
__global__ __launch_bounds__(256) void k_i8_colmax(I8QuantParams p, u32* part, float* sums, int64_t strip_rows) {
  typedef typename DT::T E;
  __shared__ u32 most[4][512];
  __shared__ float sum[SUMS ? 4 : 1][SUMS ? 512 : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 512 + 8 * lane;
  const int64_t r0 = blockIdx.y * strip_rows, r1 = min(r0 + strip_rows, p.R);
  u32 m[8] = {};
  float s[8] = {};
  const E* x = reinterpret_cast<const E*>(p.x) + c * p.sc;
#pragma unroll 4
  for (int64_t r = r0 + wave; r < r1; r += 4) {
    const Vec8<DT> v = load8_step<DT>(x + r * p.sr, 0, p.C - c, p.sc);
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const float e = elem<DT>(v, k);
      m[k] = max(m[k], __float_as_uint(e) & 0x7FFFFFFFu);
      if (SUMS) s[k] += e;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; k++) {
    most[wave][8 * lane + k] = m[k];
    if (SUMS) sum[wave][8 * lane + k] = s[k];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int64_t col = (int64_t)blockIdx.x * 512 + i;
    if (col >= p.C) continue;
    part[blockIdx.y * p.C + col] = max(max(most[0][i], most[1][i]), max(most[2][i], most[3][i]));
    if (SUMS) sums[blockIdx.y * p.C + col] = (sum[0][i] + sum[1][i]) + (sum[2][i] + sum[3][i]);
  }
}

// The strips' join: scales and their reciprocals, and the column sums. 64 columns a block, a wave for every sixteenth strip.
template <class DT, bool SUMS>
__global__ __launch_bounds__(1024) void k_i8_colscale(const u32* part, const float* sums, int strips, int64_t C, float* scales,
                                                      float* recip, typename DT::T* out) {
  __shared__ u32 most[16][64];
  __shared__ double sum[SUMS ? 16 : 1][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane, c = col < C ? col : C - 1;
  u32 m = 0;
  double s = 0;
  // eight strips requested at a time
  for (int k = wave; k < strips; k += 128) {
    u32 a[8];
    float b[SUMS ? 8 : 1];
#pragma unroll
    for (int u = 0; u < 8; u++) {
      const int64_t at = (int64_t)min(k + 16 * u, strips - 1) * C + c;  // past the last: it again, for its maximum
      a[u] = part[at];
      if (SUMS) b[u] = sums[at];
    }
#pragma unroll
    for (int u = 0; u < 8; u++) {
      m = max(m, a[u]);
      if (SUMS && k + 16 * u < strips) s += (double)b[u];
    }
  }
  most[wave][lane] = m;
  if (SUMS) sum[wave][lane] = s;
  __syncthreads();
  if (wave || col >= C) return;
#pragma unroll
  for (int w = 1; w < 16; w++) {
    m = max(m, most[w][lane]);
    if (SUMS) s += sum[w][lane];
  }
  const Scale8 q = scale8(m);
  scales[col] = q.s;
  recip[col] = q.r;
  if (SUMS) out[col] = DT::store((float)s);
}

// Codes of a tile of 64 rows x 128 columns of x as the transpose's: a thread takes four rows of eight columns, makes a word
// of four codes for each column, and the words change places in LDS. Word `rg` of column 8 lc + j lies at lc * 132 + 16 j + rg:
// a wave's 64 writes (16 lc, four rg) and 16 lanes' 16-byte reads each meet 64 distinct banks.
template <class DT>
__global__ __launch_bounds__(256) void k_i8_cols(I8QuantParams p, const float* recip, int64_t tiles_c, int64_t tiles) {
  typedef typename DT::T E;
  __shared__ __align__(16) u32 words[16 * 132];
  const int t = threadIdx.x, lc = t & 15, rg = t >> 4;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t tr = tile / tiles_c, tc = tile - tr * tiles_c;
    const int64_t c = tc * 128 + 8 * lc, r = tr * 64 + 4 * rg;
    const E* x = reinterpret_cast<const E*>(p.x) + r * p.sr + c * p.sc;
    Vec8<DT> v[4];
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = r + i < p.R ? load8_step<DT>(x + i * p.sr, 0, p.C - c, p.sc) : zero8<DT>();
    const Vec8<MxF32> rv = load8<MxF32>(recip, c, p.C), sv = load8<MxF32>(p.cols.scales, c, p.C);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float r = elem<MxF32>(rv, j), s = elem<MxF32>(sv, j);
      Code8 q[4];
      float far = 0.f;
#pragma unroll
      for (int i = 0; i < 4; i++) q[i] = code8(elem<DT>(v[i], j), s, r, far);
      if (__builtin_amdgcn_ballot_w64(border8(far, s))) {
#pragma unroll
        for (int i = 0; i < 4; i++) mend8(q[i], s);
      }
      words[lc * 132 + 16 * j + rg] = r == 0.f ? 0u : bytes4(q[0].u, q[1].u, q[2].u, q[3].u);
    }
    __syncthreads();
    // 16 columns x 64 codes are a kilobyte of the tensor: a lane stores 16 codes of one
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int i = t + 256 * h, cc = i >> 2, w4 = i & 3;
      const v4i word = *reinterpret_cast<const v4i*>(&words[(cc >> 3) * 132 + 16 * (cc & 7) + 4 * w4]);
      const int64_t col = tc * 128 + cc;
      if (col < p.C) *reinterpret_cast<v4i*>(p.cols.codes + i8_at(col, tr * 64 + 16 * w4, p.cols.kq)) = word;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------ dequantise
// 64 rows x 64 codes a block: a lane turns 16 codes into 16 neighbouring outputs.
template <class DT>
__global__ __launch_bounds__(256) void k_i8_dequantize(I8DequantParams p, int64_t tiles) {
  typedef typename DT::T E;
  const int t = threadIdx.x;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t tr = tile / p.kq, st = tile - tr * p.kq;
    const int64_t r = tr * 64 + (t >> 2), c = st * 64 + 16 * (t & 3);
    if (r >= p.rows || c >= p.K) continue;
    const v4i w = *reinterpret_cast<const v4i*>(p.codes + i8_at(r, c, p.kq));
    const float s = p.scales[r];
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; k++) v[k] = (float)(int8_t)((u32)w[k >> 2] >> (8 * (k & 3))) * s;
    E* dst = reinterpret_cast<E*>(p.out) + r * p.ldo + c;
    if (c + 16 <= p.K) {
      u32 o[DT::size * 4];
#pragma unroll
      for (int q = 0; q < DT::size * 4; q++) {
        if constexpr (DT::size == 4)
          o[q] = __float_as_uint(v[q]);
        else
          o[q] = DT::pack(v[2 * q], v[2 * q + 1]);
      }
      __builtin_memcpy(dst, o, sizeof o);
    } else {
#pragma unroll
      for (int k = 0; k < 16; k++)
        if (c + k < p.K) dst[k] = DT::store(v[k]);
    }
  }
}

}  // namespace dev

using namespace dev;

constexpr int64_t kMostBlocks = 1 << 20;  // of kernels that walk over what is left
static unsigned blocks_of(int64_t n) { return (unsigned)(n < kMostBlocks ? n : kMostBlocks); }

// Rows that are read in whole vectors.
static bool one_vector(int64_t C, int64_t sc) { return C >= 8 && sc == 1; }

template <class DT, int T, int NV>
static void launch_rows(const I8QuantParams& p, hipStream_t stream) {
  constexpr int RPB = T < 256 ? 256 / T : 1, THREADS = T < 256 ? 256 : T;
  const int64_t blocks = (p.R + RPB - 1) / RPB, most = 2048 * 256 / THREADS;  // as many as the chip holds at once
  k_i8_rows<DT, T, NV, ROWS_ALONE><<<(unsigned)(blocks < most ? blocks : most), THREADS, 0, stream>>>(p, nullptr, nullptr);
}

// Two or three vectors a thread, so that several rows are on a compute unit: 8192 x 12288 bf16 62 us with 512 threads of three, 4096 x
// 4096 11.6 with 256 of two (128 of four a third more).
template <class DT>
static hipError_t rows_t(const I8QuantParams& p, hipStream_t stream) {
  const int64_t Kp = (int64_t)p.rows.kq * 64;
  if (!one_vector(p.C, p.sc))
    launch_rows<DT, 1024, 0>(p, stream);
  else if (Kp <= 512)
    launch_rows<DT, 64, 1>(p, stream);
  else if (Kp <= 1024)
    launch_rows<DT, 64, 2>(p, stream);
  else if (Kp <= 2048)
    launch_rows<DT, 128, 2>(p, stream);
  else if (Kp <= 4096)
    launch_rows<DT, 256, 2>(p, stream);
  else if (Kp <= 8192)
    launch_rows<DT, 512, 2>(p, stream);
  else if (Kp <= 12288)
    launch_rows<DT, 512, 3>(p, stream);
  else if (Kp <= 16384)
    launch_rows<DT, 1024, 2>(p, stream);
  else
    launch_rows<DT, 1024, 0>(p, stream);
  return hipGetLastError();
}

// Rows whose codes and column maxima come from one reading: they fit a block's registers.
constexpr int64_t kSharedRow = 16384;

// Threads of a block of the kernel for both: a vector a thread, two past 4096 columns (8192 x 8192 bf16 in 512 threads of two 45 us, in 1024 of
// one 61; float32, whose registers do not hold two and their sums, 91 and 79: it takes 1024 of one). size: of an element.
static int shared_threads(int64_t C, int size) {
  const int64_t Kp = i8_kq(C) * 64;
  if (Kp <= 2048) return 256;
  return Kp <= (size == 2 ? 8192 : 4096) ? 512 : 1024;
}

// Rows that a thread adds up in float32, at most (more only where a grid would pass 65535 strips: 2^28 rows). A longer chain's error grows with
// the rows.
constexpr int64_t kChain = 1024;

// Strips of rows that a column's maximum is taken over. Read with the rows (`shared`): 256, so that every compute unit has one; more where that
// leaves each enough rows to be worth its part's way through memory, up to as many as the chip holds at once (8192 x 12288 bf16 in 128, 256, 512
// strips 140, 81 and 89 us; 777 x 5003 12.9, 10.5 and 12.6; with the join and the codes 4096 x 5000 float32 in 256 and 512 51.5 and 54.5, 2048 x
// 5000 f16 26.2 and 26.7). 1024 threads fill a unit, but those that keep one float32 vector's maxima leave room for a second block, which pays
// where a quarter of them or more has no columns (both ways in 256 and 512 strips: 20000 x 4300 202 and 178, 16384 x 6000 226 and 213, 8192 x 7000 124
// and 127, 8192 x 8192 143 and 152; with sums 8192 x 5000 122 and 130). Alone: enough blocks for the chip, of 16 rows or more.
static int64_t strips_of(int64_t R, int64_t C, bool shared, int size, bool sums) {
  int64_t strips;
  if (shared) {
    const bool two = size == 4 && !sums && i8_kq(C) * 64 <= 6144;
    const int64_t most = 256 * 1024 / shared_threads(C, two ? 2 : size), rows = i8_kq(C) <= 64 ? 4 : 16;  // of a strip, at least
    strips = R / rows < most ? R / rows : most;
    if (strips < 256) strips = R < 256 ? R : 256;
    return strips;
  }
  const int64_t chunks = (C + 511) / 512;
  strips = (2048 + chunks - 1) / chunks;
  const int64_t most = (R + 15) / 16;
  if (strips > most) strips = most;
  if (strips > 256) strips = 256;
  const int64_t least = (R + 4 * kChain - 1) / (4 * kChain);
  if (strips < least) strips = least < 65535 ? least : 65535;
  const int64_t rows = (R + strips - 1) / strips;
  return (R + rows - 1) / rows;
}

// Launches that leave so many strips each, of rows read once for their codes, maxima and sums: no sum over more than kChain rows. (More
// strips in one launch instead: 600000 x 4096 bf16 3.6 ms, not 3.3.)
static int64_t runs_of(int64_t R, int64_t strips) { return (R + strips * kChain - 1) / (strips * kChain); }

static int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// A matrix whose columns are contiguous is its transpose, with the outputs exchanged.
static bool exchanged(int64_t sr, int64_t sc) { return sr == 1 && sc != 1; }

static bool shares(int64_t C, int64_t sc, bool rows) { return rows && one_vector(C, sc) && i8_kq(C) * 64 <= kSharedRow; }

size_t i8_quantize_bytes(int64_t R, int64_t C, int64_t sr, int64_t sc, bool rows, bool cols) {
  if (exchanged(sr, sc)) {
    const int64_t r = R, s = sr;
    const bool k = rows;
    R = C, C = r, sr = sc, sc = s, rows = cols, cols = k;
  }
  if (!cols) return 0;
  const bool shared = shares(C, sc, rows);
  // 16-bit elements have as many strips as float32 ones, or more
  const int64_t strips = strips_of(R, C, shared, 2, true), parts = shared ? strips * runs_of(R, strips) : strips;
  return (size_t)(round256(C * 4) + 2 * round256(parts * C * 4));
}

bool i8_quantize_fits(int64_t R, int64_t C, int64_t sr, int64_t sc, bool rows, bool cols) {
  const bool swap = exchanged(sr, sc);
  return !(swap ? rows : cols) || mx_fits_grid(((swap ? R : C) + 63) / 64, 1024);
}

template <class DT, int T, int NV>
static void launch_shared(const I8QuantParams& p, int64_t strips, u32* part, float* sums, hipStream_t stream) {
  const int64_t runs = runs_of(p.R, strips), rows = ((p.R + runs - 1) / runs + 15) / 16 * 16;  // whole tiles of codes
  if (p.sums)
    for (int64_t k = 0; k < runs; k++) {
      I8QuantParams q = p;
      q.x = reinterpret_cast<const typename DT::T*>(p.x) + k * rows * p.sr;
      q.rows.codes += k * (rows >> 4) * p.rows.kq * 1024;
      q.rows.scales += k * rows;
      q.R = min(rows, p.R - k * rows);
      k_i8_rows<DT, T, NV, ROWS_MAXIMA_AND_SUMS><<<(unsigned)strips, T, 0, stream>>>(q, part + k * strips * p.C, sums + k * strips * p.C);
    }
  else
    k_i8_rows<DT, T, NV, ROWS_AND_MAXIMA><<<(unsigned)strips, T, 0, stream>>>(p, part, sums);
}

template <class DT>
static hipError_t cols_t(const I8QuantParams& p, hipStream_t stream) {
  const bool shared = shares(p.C, p.sc, p.rows.codes != nullptr);
  const int64_t strips = strips_of(p.R, p.C, shared, DT::size, p.sums != nullptr);
  float* recip = reinterpret_cast<float*>(p.workspace);
  u32* part = reinterpret_cast<u32*>((uint8_t*)p.workspace + round256(p.C * 4));
  const int64_t parts = shared && p.sums ? strips * runs_of(p.R, strips) : strips;
  float* sums = reinterpret_cast<float*>((uint8_t*)part + round256(parts * p.C * 4));
  if (shared) {
    switch (shared_threads(p.C, DT::size)) {
      case 256: launch_shared<DT, 256, 1>(p, strips, part, sums, stream); break;
      case 512:
        if constexpr (DT::size == 2)
          if (p.rows.kq > 64) {
            launch_shared<DT, 512, 2>(p, strips, part, sums, stream);
            break;
          }
        launch_shared<DT, 512, 1>(p, strips, part, sums, stream);
        break;
      default:
        if constexpr (DT::size == 4)
          if (p.rows.kq <= 128) {
            launch_shared<DT, 1024, 1>(p, strips, part, sums, stream);
            break;
          }
        launch_shared<DT, 1024, 2>(p, strips, part, sums, stream);
    }
  } else {
    const int64_t strip_rows = (p.R + strips - 1) / strips;
    const dim3 grid((unsigned)((p.C + 511) / 512), (unsigned)strips);
    if (p.sums)
      k_i8_colmax<DT, true><<<grid, 256, 0, stream>>>(p, part, sums, strip_rows);
    else
      k_i8_colmax<DT, false><<<grid, 256, 0, stream>>>(p, part, sums, strip_rows);
  }
  const unsigned joins = (unsigned)((p.C + 63) / 64);
  if (!p.sums)
    k_i8_colscale<MxF32, false><<<joins, 1024, 0, stream>>>(part, sums, (int)parts, p.C, p.cols.scales, recip, nullptr);
  else if (p.sums_dtype == SVDQ_F32)
    k_i8_colscale<MxF32, true><<<joins, 1024, 0, stream>>>(part, sums, (int)parts, p.C, p.cols.scales, recip, (float*)p.sums);
  else if (p.sums_dtype == SVDQ_BF16)
    k_i8_colscale<MxBF16, true><<<joins, 1024, 0, stream>>>(part, sums, (int)parts, p.C, p.cols.scales, recip, (uint16_t*)p.sums);
  else
    k_i8_colscale<MxF16, true><<<joins, 1024, 0, stream>>>(part, sums, (int)parts, p.C, p.cols.scales, recip, (uint16_t*)p.sums);
  // the transpose's stages come in pairs, so the last tile of rows may hold nothing but padding
  const int64_t tiles_c = (p.C + 127) / 128, tiles = (int64_t)p.cols.kq * tiles_c;
  k_i8_cols<DT><<<blocks_of(tiles), 256, 0, stream>>>(p, recip, tiles_c, tiles);
  return hipGetLastError();
}

template <class DT>
static hipError_t quantize_t(const I8QuantParams& p0, hipStream_t stream) {
  I8QuantParams p = p0;
  if (exchanged(p.sr, p.sc)) p.R = p0.C, p.C = p0.R, p.sr = p0.sc, p.sc = p0.sr, p.rows = p0.cols, p.cols = p0.rows;
  if (p.rows.codes && !(p.cols.codes && shares(p.C, p.sc, true))) {
    const hipError_t e = rows_t<DT>(p, stream);
    if (e != hipSuccess) return e;
  }
  return p.cols.codes ? cols_t<DT>(p, stream) : hipSuccess;
}

hipError_t launch_i8_quantize(const I8QuantParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case SVDQ_F32: return quantize_t<MxF32>(p, stream);
    case SVDQ_BF16: return quantize_t<MxBF16>(p, stream);
    default: return quantize_t<MxF16>(p, stream);
  }
}

hipError_t launch_i8_dequantize(const I8DequantParams& p, int dtype, hipStream_t stream) {
  const int64_t tiles = (p.rows + 63) / 64 * p.kq;
  switch (dtype) {
    case SVDQ_F32: k_i8_dequantize<MxF32><<<blocks_of(tiles), 256, 0, stream>>>(p, tiles); break;
    case SVDQ_BF16: k_i8_dequantize<MxBF16><<<blocks_of(tiles), 256, 0, stream>>>(p, tiles); break;
    default: k_i8_dequantize<MxF16><<<blocks_of(tiles), 256, 0, stream>>>(p, tiles);
  }
  return hipGetLastError();
}

}  // namespace svdq
