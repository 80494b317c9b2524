// Elementwise kernels on MXFP4 tensors for gfx950:
//   * k_mx_quantize    Q(x) and / or Q(x^T) of a matrix, one pass over it;
//   * k_mx_dequantize  the values of a tensor;
//   * k_mx_gated_grad  the gradients of a gated block's pre-activations, quantised both ways.
//
// Q takes 32 elements along the axis a product sums over, the smallest e with max|x| <= 6 * 2^e,
// and the E2M1 codes of x / 2^e (nearest, ties to the even code). Both are decided by exact
// operations: the maximum, a comparison of its bits, and a conversion that divides by a power of
// two. All three kernels move a few bytes per element and are bound by memory.
//
// Quantising along both axes takes one read of x: a block owns a 128 x 128 tile, quantises its
// rows from registers (a row's 32-element block is four neighbouring lanes' 8 elements each), and
// its columns from a copy of the tile in LDS (a lane reads the 32 rows of its column). 128 x 128 is
// the smallest tile whose codes fill whole 64-byte rows of the 1 KB code tiles in both directions.
#include <type_traits>

#include "mx.h"
#include "mx_device.h"
#include "mx_rows.h"

namespace svdq {
namespace dev {

constexpr int kTile = 128, kMxBlock = 32;

// Quantises a column's 32 elements (block `kb` of a stage of the transpose) held by a lane: N words of pairs or
// values. lc: column in the group.
template <class DT, int N>
__device__ inline void put_col(const MxGroup& o, const u32 (&w)[N], u32 lc, u32 kb, bool live) {
  const u32 byte = mx_scale_byte(amax_bits<DT>(w));
  v4i c;
#pragma unroll
  for (int q = 0; q < 4; q++) c[q] = (int)codes8<DT>(w + N / 4 * q, byte);
  if (!live) return;
  *reinterpret_cast<v4i*>(o.codes + ((lc << 6) + (kb << 4))) = c;
  o.scales[(lc << 2) + kb] = (uint8_t)byte;
}

// Pair of columns `pr` of 32 rows of 16-bit values in LDS (W words a row from `rows`, the pair at word `at`): the low halves
// of a lane's words, then the high halves. The tile's first 16-column group is group0; the rows are block kb of `stage`; `left` columns exist.
template <class DT>
__device__ __forceinline__ void pair_cols(const u32* rows, int W, int at, int pr, const MxOut& out, int64_t group0, int stage,
                                          int kb, int64_t left) {
  u32 lo[16], hi[16];
#pragma unroll
  for (int r = 0; r < 16; r++) {
    const u32 a = rows[2 * r * W + at], b = rows[(2 * r + 1) * W + at];
    lo[r] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    hi[r] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  }
  const MxGroup o = group_of(out, group0 + (pr >> 3), stage);
  put_col<DT>(o, lo, (2 * pr) & 15, kb, 2 * pr < left);
  put_col<DT>(o, hi, (2 * pr + 1) & 15, kb, 2 * pr + 1 < left);
}

// ------------------------------------------------------------------------------ quantise
// Block: 256 threads, a tile of 16 NP rows of 128 columns; thread t holds elements [8 (t % 16), + 8) of rows t / 16 + 16 i.
//
// The tile's LDS copy has W words per row. A column reader's lanes are 16 columns x 4 blocks of 32 rows; moving a
// row's 16-word groups by its block's number (tile_word) puts the four blocks on different banks.
template <int W>
__device__ inline int tile_word(int row, int word) {
  return row * W + (word ^ (((row >> 5) & 3) << 4));
}

template <class DT, int NP, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void k_mx_quantize(MxQuantParams p, int tiles_c) {
  constexpr int TH = 16 * NP, W = kTile * DT::size / 4;  // tile rows, words per tile row
  __shared__ __align__(16) u32 tile[COLS ? TH * W : 4];
  typedef typename DT::T T;
  const int t = threadIdx.x, l16 = t & 15, lr = t >> 4;
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int64_t c0 = (int64_t)tc * kTile + 8 * l16;
  const T* x = reinterpret_cast<const T*>(p.x) + ((int64_t)tr * TH + lr) * p.sr + c0 * p.sc;
  // rows and elements of this thread's part that exist
  const int64_t left_r = p.R - (int64_t)tr * TH, left_c = p.C - c0;

  Vec8<DT> v[NP];
#pragma unroll
  for (int i = 0; i < NP; i++) {
    v[i] = zero8<DT>();
    if (lr + 16 * i >= left_r) continue;
    const T* src = x + (int64_t)(16 * i) * p.sr;
    if (p.sc == 1) {
      v[i] = load8<DT>(src, 0, left_c);
    } else {
#pragma unroll
      for (int q = 0; q < 8; q++) {
        if (q >= left_c) continue;
        const T e = src[q * p.sc];
        if constexpr (DT::size == 4)
          v[i].w[q] = __float_as_uint(e);
        else
          v[i].w[q >> 1] |= (u32)e << (16 * (q & 1));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NP; i++) {
    if (!COLS && 16 * i >= left_r) break;
    if constexpr (ROWS) put_row<DT>(group_of(p.rows, (int64_t)tr * NP + i, tc), v[i], lr, 8 * l16, lr + 16 * i < left_r);
    if constexpr (COLS) {
#pragma unroll
      for (int h = 0; h < DT::size / 2; h++)
        *reinterpret_cast<v4i*>(&tile[tile_word<W>(lr + 16 * i, l16 * 2 * DT::size + 4 * h)]) =
            v4i{(int)v[i].w[4 * h], (int)v[i].w[4 * h + 1], (int)v[i].w[4 * h + 2], (int)v[i].w[4 * h + 3]};
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    // sixteen lanes take 16 columns, or 16 pairs of them, of one block of 32 rows
    constexpr int KB = TH / 32, PER = kTile / TH;  // blocks in the tile, tiles in a stage
    constexpr int GROUPS = W / 16, AT_ONCE = 16 / KB;
    const int s16 = t >> 4, kb = s16 % KB, stage = tr / PER, at_kb = tr % PER * KB + kb;
    const u32* rows = tile + 32 * kb * W;
    const int64_t left = p.C - (int64_t)tc * kTile;
#pragma unroll
    for (int h = 0; h < (GROUPS + AT_ONCE - 1) / AT_ONCE; h++) {
      const int w = s16 / KB + AT_ONCE * h, c = 16 * w + l16, at = c ^ (kb << 4);  // a block's rows share their move
      if (w >= GROUPS) continue;
      if constexpr (DT::size == 4) {
        u32 e[32];
#pragma unroll
        for (int r = 0; r < 32; r++) e[r] = rows[r * W + at];
        put_col<DT>(group_of(p.cols, (int64_t)tc * 8 + w, stage), e, l16, at_kb, c < left);
      } else {
        pair_cols<DT>(rows, W, at, c, p.cols, (int64_t)tc * 8, stage, at_kb, left);
      }
    }
  }
}

// ------------------------------------------------------------------------------ dequantise
// Block: 256 threads, 64 rows x one stage; a lane turns 8 codes into 8 neighbouring outputs.
template <class DT>
__global__ __launch_bounds__(256) void k_mx_dequantize(MxDequantParams p, int stages) {
  typedef typename DT::T T;
  const int t = threadIdx.x, l16 = t & 15;
  const int64_t tr = blockIdx.x / stages;
  const int st = (int)(blockIdx.x - tr * stages);
  const int64_t c = (int64_t)st * kTile + 8 * l16;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t r = tr * 64 + (t >> 4) + 16 * i;
    if (r >= p.rows || c >= p.K) continue;
    const u32 w = *reinterpret_cast<const u32*>(p.codes + (((r >> 4) * p.kq + st) << 10) + ((r & 15) << 6) + l16 * 4);
    const u32 byte = p.scales[mx_scale_tiled_index(r, 4 * st + (l16 >> 2), p.kq)];
    const float s = byte == 255u ? __uint_as_float(0x7FC00000u) : mx_scale_value(byte);
    float v[8];
#define MX_PAIR(Q)                                                                \
  {                                                                               \
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, Q);          \
    v[2 * Q] = d[0] * s;                                                          \
    v[2 * Q + 1] = d[1] * s;                                                      \
  }
    MX_PAIR(0) MX_PAIR(1) MX_PAIR(2) MX_PAIR(3)
#undef MX_PAIR
    T* dst = reinterpret_cast<T*>(p.out) + r * p.ldo + c;
    if (c + 8 <= p.K) {
      u32 o[DT::size * 2];
#pragma unroll
      for (int q = 0; q < DT::size * 2; q++) {
        if constexpr (DT::size == 4)
          o[q] = __float_as_uint(v[q]);
        else
          o[q] = DT::pack(v[2 * q], v[2 * q + 1]);
      }
      __builtin_memcpy(dst, o, sizeof o);
    } else {
#pragma unroll
      for (int q = 0; q < 8; q++)
        if (c + q < p.K) dst[q] = DT::store(v[q]);
    }
  }
}

// ------------------------------------------------------------------------------ gated gradients
// A gradient v of known error bound err is as good as the formula's in binary64 for every code and
// block maximum when no border lies within err of it. The borders between E2M1 values are 0.25,
// 0.75, 1.25, 1.75, 2.5, 3.5 and 5 times a power of two, and a block's exponent changes at 1.5
// times one: all have 0 in the low 21 bits of their float32 pattern. So v is settled when |v| - err
// and |v| + err agree in the bits above those. An unsettled v (about one in 20000 for pre-activations
// of unit scale) is computed in binary64.
//
// What a gradient is quantised from, in either direction, is 16 bits of it: those of a bfloat16 cut off toward
// zero, with the lowest bit set if anything was cut off. That lies on the same side of every border as v does.
// A settled v lies on no border, so its bit is simply set; and the tile's copy in LDS takes half the room.
//
// Instructions bound this kernel as much as memory does (about 45 for each pair dg, du): two elements are
// tested together, by the bits in which any of their ends differ, and eight by their least tail (see ActValue).
constexpr u32 kOpen = 1u << 21;
__device__ __forceinline__ u32 ends_differ(float v, float err) {
  const float a = fabsf(v);
  return __float_as_uint(a - err) ^ __float_as_uint(a + err);
}

// The 16 bits for a binary64 gradient (from infinity on, any of those mark a block).
__device__ inline u32 to_odd16(double v) {
  const float f = (float)v;
  u32 u = __float_as_uint(f);
  const double d = (double)f;
  if (!(fabs(v) < 0x1p128) || d == v) return (u >> 16) | ((u & 0xFFFFu) ? 1u : 0u);
  if (fabs(d) > fabs(v)) u -= 1;  // toward zero (f is not zero then; it may be the infinity above the largest float)
  return (u >> 16) | (v < 0 ? 0x8001u : 1u);
}

// Entry q of a register array by selects. (As a loop over constants the compiler turns them into an index, and the
// array into memory.)
template <int N, int K = 0>
__device__ __forceinline__ u32 get_at(const u32 (&w)[N], int q) {
  const u32 e = w[K];
  if constexpr (K + 1 < N) {
    const u32 rest = get_at<N, K + 1>(w, q);
    return q == K ? e : rest;
  } else {
    return e;
  }
}
template <int N, int K = 0>
__device__ __forceinline__ void set_at(u32 (&w)[N], int q, u32 v) {
  const u32 e = w[K];
  w[K] = q == K ? v : e;
  if constexpr (K + 1 < N) set_at<N, K + 1>(w, q, v);
}

template <class DT>
__device__ __forceinline__ float pick(const Vec8<DT>& v, int q) {
  if constexpr (DT::size == 4)
    return __uint_as_float(get_at(v.w, q));
  else
    return DT::load((uint16_t)(get_at(v.w, q >> 1) >> (16 * (q & 1))));
}
__device__ __forceinline__ void set16(Vec8<MxBF16>& o, int q, u32 v) {
  const u32 w = get_at(o.w, q >> 1);
  set_at(o.w, q >> 1, q & 1 ? (w & 0xFFFFu) | (v << 16) : (w & 0xFFFF0000u) | v);
}

// The cut-off halves of two settled gradients.
__device__ __forceinline__ u32 odd_pair(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u) | 0x00010001u;
}

template <class DT>
struct GradIn {
  Vec8<DT> dh, g, u;
};

// Eight elements of dg and / or du (whichever of GATE and UP) in those 16 bits.
template <class DT, int ACT, bool GATE, bool UP>
__device__ __forceinline__ void grad8(const GradIn<DT>& x, Vec8<MxBF16>& dg, Vec8<MxBF16>& du) {
  u32 differ[4];
  float tail = 0.f, reach = 0.f;
#pragma unroll
  for (int h = 0; h < 4; h++) {
    float vg[2], vu[2];
    differ[h] = 0;
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const float dh = elem<DT>(x.dh, 2 * h + k);
      const ActValue<float> r = act_value<ACT, float>(elem<DT>(x.g, 2 * h + k));
      tail = r.tail < tail ? r.tail : tail;
      if (GATE) {
        const float a = dh * elem<DT>(x.u, 2 * h + k);
        if (DT::wide) reach += fabsf(a);
        vg[k] = a * r.d;
        differ[h] |= ends_differ(vg[k], fabsf(a) * r.abs_d);
      }
      if (UP) {
        vu[k] = dh * r.a;
        differ[h] |= ends_differ(vu[k], fabsf(vu[k]) * r.ew);
      }
    }
    if (GATE) dg.w[h] = odd_pair(vg[0], vg[1]);
    if (UP) du.w[h] = odd_pair(vu[0], vu[1]);
  }
  // an infinite dh * u: times a derivative of 0 it is a NaN, whose two ends agree, though the formula's value may be finite
  const bool far = tail < -60.f || !(reach < __builtin_inff());
  if (!((differ[0] >= kOpen) | (differ[1] >= kOpen) | (differ[2] >= kOpen) | (differ[3] >= kOpen) | far)) return;
#pragma unroll 1
  for (int q = 0; q < 8; q++) {
    if (get_at(differ, q >> 1) < kOpen && !far) continue;
    const double dh = (double)pick<DT>(x.dh, q);
    const ActValue<double> e = act_value<ACT, double>((double)pick<DT>(x.g, q));
    if (GATE) set16(dg, q, to_odd16((dh * (double)pick<DT>(x.u, q)) * e.d));
    if (UP) set16(du, q, to_odd16(dh * e.a));
  }
}

// A tile of 32 rows (one block of the transpose) of 64 columns by 256 threads, thread t with elements [8 (t % 8), + 8) of row
// t / 8. Many small blocks hide each other's loads: tiles of 128 rows, whose columns' codes fill whole 64-byte rows, were
// no faster at 4096 x 12288 (103 us against 105) and twice as slow at 515 x 2731 (24 us against 11.7).
// GRAD_PAIR: columns [c0, c0 + 64) of dh, g and u give a tile of dg and one of du. GRAD_GATE, GRAD_UP, GRAD_MIXED: a tile of
// d = [dg | du] at j0, all dg, all du, or some of either.
constexpr int kGradRows = 32, kGradCols = 64;
enum { GRAD_PAIR, GRAD_GATE, GRAD_UP, GRAD_MIXED };

template <class DT, int ACT, int MODE, bool ROWS, bool COLS>
__device__ __forceinline__ void grad_tile(const MxGradParams& p, u32* tile, int tr, int tc) {
  constexpr int LPR = kGradCols / 8, W = kGradCols / 2, TILE = kGradRows * W;  // lanes and words per row, words of a tile
  typedef typename DT::T T;
  const int t = threadIdx.x, lc = t % LPR, lr = t / LPR;
  const int half = __builtin_amdgcn_readfirstlane(t >> 7);  // the 16-row half
  const int64_t F = p.F, row = (int64_t)tr * kGradRows + lr;
  const int64_t j = (int64_t)tc * kGradCols + 8 * lc, c = MODE == GRAD_UP || (MODE == GRAD_MIXED && j >= F) ? j - F : j;
  Vec8<MxBF16> d = zero8<MxBF16>(), du = zero8<MxBF16>();
  if (row < p.M) {
    GradIn<DT> x{zero8<DT>(), zero8<DT>(), zero8<DT>()};
    const T* dr = reinterpret_cast<const T*>(p.dh) + row * p.ldh;
    const T* gr = reinterpret_cast<const T*>(p.gu) + row * p.ldgu;
    if (MODE != GRAD_MIXED || j >= F || j + 8 <= F) {
      x.dh = load8<DT>(dr, c, F);
      x.g = load8<DT>(gr, c, F);
      if (MODE != GRAD_UP) x.u = load8<DT>(gr + F, c, F);
    } else {
#pragma unroll
      for (int q = 0; q < 8; q++) {
        if (j + q >= 2 * F) continue;
        const int64_t e = j + q < F ? j + q : j + q - F;
        if constexpr (DT::size == 4) {
          x.dh.w[q] = __float_as_uint(dr[e]);
          x.g.w[q] = __float_as_uint(gr[e]);
          x.u.w[q] = __float_as_uint(gr[F + e]);
        } else {
          x.dh.w[q >> 1] |= (u32)dr[e] << (16 * (q & 1));
          x.g.w[q >> 1] |= (u32)gr[e] << (16 * (q & 1));
          x.u.w[q >> 1] |= (u32)gr[F + e] << (16 * (q & 1));
        }
      }
    }
    if constexpr (MODE == GRAD_UP)
      grad8<DT, ACT, false, true>(x, du, d);
    else
      grad8<DT, ACT, true, MODE != GRAD_GATE>(x, d, du);
    if constexpr (MODE == GRAD_MIXED) {
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const u32 from_up = (j + 2 * q >= F ? 0xFFFFu : 0u) | (j + 2 * q + 1 >= F ? 0xFFFF0000u : 0u);
        d.w[q] = (d.w[q] & ~from_up) | (du.w[q] & from_up);
      }
    }
  }
  if constexpr (ROWS) {
    // places in a row of the row tensor: the tile's, and du's (F is a multiple of 32, not of a stage)
    constexpr int PER = kTile / kGradCols;
    const int64_t group = (int64_t)tr * 2 + half, up_at = F + (int64_t)tc * kGradCols;
    const bool live = row < p.M && (MODE != GRAD_PAIR || c < F);
    put_row<MxBF16>(group_of(p.rows, group, tc / PER), d, lr & 15, (tc % PER) * kGradCols + 8 * lc, live);
    if constexpr (MODE == GRAD_PAIR)
      put_row<MxBF16>(group_of(p.rows, group, up_at / kTile), du, lr & 15, (u32)(up_at % kTile) + 8 * lc, live);
  }
  if constexpr (COLS) {
    // two copies of 32 rows; a reader's lanes are 16 pairs of columns of one of them
    *reinterpret_cast<v4i*>(&tile[lr * W + 4 * lc]) = v4i{(int)d.w[0], (int)d.w[1], (int)d.w[2], (int)d.w[3]};
    if constexpr (MODE == GRAD_PAIR)
      *reinterpret_cast<v4i*>(&tile[TILE + lr * W + 4 * lc]) = v4i{(int)du.w[0], (int)du.w[1], (int)du.w[2], (int)du.w[3]};
    __syncthreads();
    const int64_t col0 = (int64_t)tc * kGradCols;
    const int side = t >> 5, pr = t & 31;
    if (side < (MODE == GRAD_PAIR ? 2 : 1))
      pair_cols<MxBF16>(tile + side * TILE, W, pr, pr, p.cols, (col0 + (side ? F : 0)) / 16, tr / (kTile / kGradRows),
                        tr % (kTile / kGradRows), (MODE == GRAD_PAIR ? F : 2 * F) - col0);
  }
}

// F a multiple of 32, so that blocks along d = [dg | du] belong to one side: every input is read once.
template <class DT, int ACT, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void k_mx_gated_grad(MxGradParams p, int tiles_c) {
  __shared__ __align__(16) u32 tile[COLS ? kGradRows * kGradCols : 4];
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  grad_tile<DT, ACT, GRAD_PAIR, ROWS, COLS>(p, tile, tr, tc);
  if constexpr (ROWS) {
    // the row tensor's padding past 2 F, zero codes and bytes, by the last column of blocks
    if (tc == tiles_c - 1) {
      const int l16 = threadIdx.x & 15;
      for (int st = (int)(2 * p.F / kTile); st < p.rows.kq; st++) {
        const bool past = (int64_t)st * kTile + 8 * l16 >= 2 * p.F;
        for (int r = threadIdx.x >> 4; r < kGradRows; r += 16) {
          const int64_t row = (int64_t)tr * kGradRows + r;
          put_row<MxBF16>(group_of(p.rows, row >> 4, st), zero8<MxBF16>(), row & 15, 8 * l16, past && row < p.M);
        }
      }
    }
  }
}

// Any F: tiles of d itself. The two that read the same dh and g, one on either side of F, go to blocks 8 apart:
// neighbours on one XCD, so that the second finds them in its L2.
template <class DT, int ACT, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void k_mx_gated_grad_any(MxGradParams p, int tiles_c, int pairs) {
  __shared__ __align__(16) u32 tile[COLS ? kGradRows * kGradCols / 2 : 4];
  const int64_t id = (int64_t)(blockIdx.x >> 4) * 8 + (blockIdx.x & 7);
  const int tr = (int)(id / pairs), pair = (int)(id - (int64_t)tr * pairs), side = (blockIdx.x >> 3) & 1;
  const int first_up = (int)(p.F / kGradCols), tc = side ? first_up + pair : pair;
  if (side ? tc >= tiles_c : tc >= first_up) return;
  if (COLS ? tr >= p.cols.kq * (kTile / kGradRows) : (int64_t)tr * kGradRows >= p.M) return;
  if (side == 0)
    grad_tile<DT, ACT, GRAD_GATE, ROWS, COLS>(p, tile, tr, tc);
  else if (pair != 0)
    grad_tile<DT, ACT, GRAD_UP, ROWS, COLS>(p, tile, tr, tc);
  else
    grad_tile<DT, ACT, GRAD_MIXED, ROWS, COLS>(p, tile, tr, tc);
}

}  // namespace dev

using namespace dev;

// Calls f(storage type) for a dtype checked by the caller.
template <class Fn>
static hipError_t with_dtype(int dtype, Fn f) {
  switch (dtype) {
    case SVDQ_F32: return f(MxF32());
    case SVDQ_BF16: return f(MxBF16());
    default: return f(MxF16());
  }
}

static int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

// Tiles of 128 rows, whose columns' codes fill whole 64-byte rows, while they fill the chip, else of 32 rows. Measured,
// bf16, both directions: 8192 x 12288 59 us (80 with tiles of 32 x 64), 2048 x 4096 7.9 us with 32 rows against 8.7, 777 x
// 5003 6.2 against 8.4.
constexpr int64_t kFewTiles = 768;

struct QuantGrid {
  MxQuantParams p;
  bool few;
  int64_t tc, blocks;
};
static QuantGrid quant_grid(const MxQuantParams& p0) {
  QuantGrid g{p0, false, 0, 0};
  MxQuantParams& p = g.p;
  if (p.sc != 1 && p.sr == 1) {  // columns are contiguous: the transpose's rows
    const MxQuantParams q = p;
    p.R = q.C, p.C = q.R, p.sr = q.sc, p.sc = q.sr, p.rows = q.cols, p.cols = q.rows;
  }
  g.few = tiles_of(p.R) * tiles_of(p.C) < kFewTiles;
  const int64_t th = g.few ? 32 : kTile;
  // a direction that is written covers its padding too
  g.tc = p.rows.codes ? p.rows.kq : tiles_of(p.C);
  g.blocks = g.tc * (p.cols.codes ? (int64_t)p.cols.kq * (kTile / th) : (p.R + th - 1) / th);
  return g;
}

bool mx_quantize_fits(const MxQuantParams& p) { return mx_fits_grid(quant_grid(p).blocks, 256); }

template <class DT, int NP, bool ROWS, bool COLS>
static hipError_t launch_quant(const QuantGrid& g, hipStream_t stream) {
  k_mx_quantize<DT, NP, ROWS, COLS><<<dim3((unsigned)g.blocks), 256, 0, stream>>>(g.p, (int)g.tc);
  return hipGetLastError();
}

hipError_t launch_mx_quantize(const MxQuantParams& p, int dtype, hipStream_t stream) {
  const QuantGrid g = quant_grid(p);
  if (!mx_fits_grid(g.blocks, 256)) return hipErrorInvalidConfiguration;
  return with_dtype(dtype, [&](auto d) {
    typedef decltype(d) DT;
    if (g.p.rows.codes && g.p.cols.codes)
      return g.few ? launch_quant<DT, 2, true, true>(g, stream) : launch_quant<DT, 8, true, true>(g, stream);
    if (g.p.rows.codes) return g.few ? launch_quant<DT, 2, true, false>(g, stream) : launch_quant<DT, 8, true, false>(g, stream);
    return g.few ? launch_quant<DT, 2, false, true>(g, stream) : launch_quant<DT, 8, false, true>(g, stream);
  });
}

hipError_t launch_mx_dequantize(const MxDequantParams& p, int dtype, hipStream_t stream) {
  const int64_t st = tiles_of(p.K), blocks = (p.rows + 63) / 64 * st;
  if (!mx_fits_grid(blocks, 256)) return hipErrorInvalidConfiguration;
  return with_dtype(dtype, [&](auto d) {
    k_mx_dequantize<decltype(d)><<<dim3((unsigned)blocks), 256, 0, stream>>>(p, (int)st);
    return hipGetLastError();
  });
}

// Measured at 4096 rows, bf16, silu, both directions: 106 us for F = 12288 as pairs, 152 us for F = 12300.
struct GradGrid {
  bool pairs;  // dg's and du's tiles of the same columns in one block
  int64_t tc, across, blocks;
};
static GradGrid grad_grid(const MxGradParams& p) {
  GradGrid g{p.F % kMxBlock == 0, 0, 0, 0};
  const int64_t tr = p.cols.codes ? (int64_t)p.cols.kq * (kTile / kGradRows) : (p.M + kGradRows - 1) / kGradRows;
  if (g.pairs) {
    g.tc = (p.F + kGradCols - 1) / kGradCols;
    g.blocks = g.tc * tr;
  } else {
    // tiles of [0, 2F), with the row tensor's padding; those that begin below F, and those from the one that holds F on
    g.tc = p.rows.codes ? (int64_t)p.rows.kq * (kTile / kGradCols) : (2 * p.F + kGradCols - 1) / kGradCols;
    const int64_t below = p.F / kGradCols;
    g.across = g.tc - below > below ? g.tc - below : below;
    g.blocks = (g.across * tr + 7) / 8 * 16;
  }
  return g;
}

bool mx_gated_grad_fits(const MxGradParams& p) { return mx_fits_grid(grad_grid(p).blocks, 256); }

template <class DT, int ACT, bool ROWS, bool COLS>
static hipError_t launch_grad_t(const MxGradParams& p, hipStream_t stream) {
  const GradGrid g = grad_grid(p);
  if (!mx_fits_grid(g.blocks, 256)) return hipErrorInvalidConfiguration;
  if (g.pairs)
    k_mx_gated_grad<DT, ACT, ROWS, COLS><<<dim3((unsigned)g.blocks), 256, 0, stream>>>(p, (int)g.tc);
  else
    k_mx_gated_grad_any<DT, ACT, ROWS, COLS><<<dim3((unsigned)g.blocks), 256, 0, stream>>>(p, (int)g.tc, (int)g.across);
  return hipGetLastError();
}

template <class DT, int ACT>
static hipError_t launch_grad_act(const MxGradParams& p, hipStream_t stream) {
  if (p.rows.codes && p.cols.codes) return launch_grad_t<DT, ACT, true, true>(p, stream);
  return p.rows.codes ? launch_grad_t<DT, ACT, true, false>(p, stream) : launch_grad_t<DT, ACT, false, true>(p, stream);
}

hipError_t launch_mx_gated_grad(const MxGradParams& p, int dtype, hipStream_t stream) {
  return with_dtype(dtype, [&](auto d) {
    typedef decltype(d) DT;
    switch (p.act) {
      case SVDQ_ACT_SILU: return launch_grad_act<DT, SVDQ_ACT_SILU>(p, stream);
      case SVDQ_ACT_GELU: return launch_grad_act<DT, SVDQ_ACT_GELU>(p, stream);
      case SVDQ_ACT_GELU_TANH: return launch_grad_act<DT, SVDQ_ACT_GELU_TANH>(p, stream);
      default: return launch_grad_act<DT, SVDQ_ACT_RELU>(p, stream);
    }
  });
}

}  // namespace svdq
