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

namespace svdq {
namespace dev {

constexpr int kTile = 128, kMxBlock = 32;
constexpr int kGradCols = 64, kGradFew = 1024;

__device__ inline u32 quad_max(u32 v) {
  v = max(v, (u32)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // quad_perm [1,0,3,2]
  v = max(v, (u32)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // quad_perm [2,3,0,1]
  return v;
}

// The places of a 16-row group's codes and scales in a stage: uniform bases, so that a lane needs a 32-bit offset.
struct MxGroup {
  uint8_t* codes;
  uint8_t* scales;
};
__device__ inline MxGroup group_of(const MxOut& o, int64_t rows16, int64_t stage) {
  return {o.codes + ((rows16 * o.kq + stage) << 10),
          o.scales + (((rows16 >> 2) * o.kq + stage) << 8) + ((rows16 & 3) << 6)};
}

// Quantises a row's eight elements per lane: four lanes 4 j .. 4 j + 3 hold one block. lr: row in the group; pos: the
// lane's first element in the stage, a multiple of 8 (and of 32 in the first lane of a block); it may run into the next
// stages.
template <class DT>
__device__ inline void put_row(const MxGroup& o, const Vec8<DT>& v, u32 lr, u32 pos, bool live) {
  const u32 byte = mx_scale_byte(quad_max(amax_bits<DT>(v.w)));
  const u32 word = codes8<DT>(v.w, byte);
  if (!live) return;
  *reinterpret_cast<u32*>(o.codes + ((pos >> 7 << 10) + (lr << 6) + ((pos & 127) >> 1))) = word;
  if ((pos & 31) == 0) o.scales[(pos >> 7 << 8) + (lr << 2) + ((pos >> 5) & 3)] = (uint8_t)byte;
}

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

// LDS copy of a tile: W words per row. A column reader's lanes are 16 columns x 4 blocks of 32 rows; moving a row's
// 16-word groups by its block's number puts the four blocks on different banks (W = 32 has two groups: there the
// upper blocks' neighbouring rows change places).
template <int W>
__device__ inline int tile_word(int row, int word) {
  if constexpr (W == 32)
    return (row ^ ((row >> 6) & 1)) * W + (word ^ (((row >> 5) & 1) << 4));
  else
    return row * W + (word ^ (((row >> 5) & 3) << 4));
}

// Columns of a tile of 128 rows of W pairs of 16-bit values, by W / 16 waves: a lane takes a pair of columns, the low halves of its words
// and then the high halves; a wave's 16 pairs are two 16-column groups, the first of the tile being group0. `left`: columns
// that exist.
template <class DT, int W>
__device__ __forceinline__ void pair_cols(const u32* tile, const MxOut& out, int64_t group0, int stage, int wave, int l16,
                                          int kb, int at_kb, int64_t left) {
  const int pr = 16 * wave + l16;
  u32 lo[16], hi[16];
#pragma unroll
  for (int r = 0; r < 16; r++) {
    const u32 a = tile[tile_word<W>(32 * kb + 2 * r, pr)], b = tile[tile_word<W>(32 * kb + 2 * r + 1, pr)];
    lo[r] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    hi[r] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  }
  const MxGroup o = group_of(out, group0 + 2 * wave + (l16 >> 3), stage);
  put_col<DT>(o, lo, (2 * pr) & 15, at_kb, 2 * pr < left);
  put_col<DT>(o, hi, (2 * pr + 1) & 15, at_kb, 2 * pr + 1 < left);
}

// ------------------------------------------------------------------------------ quantise
// Block: 256 threads; thread t holds elements [8 (t % 16), + 8) of rows t / 16 + 16 i.
template <class DT, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void k_mx_quantize(MxQuantParams p, int tiles_c) {
  constexpr int W = kTile * DT::size / 4;  // words per tile row
  __shared__ __align__(16) u32 tile[COLS ? kTile * W : 4];
  typedef typename DT::T T;
  const int t = threadIdx.x, l16 = t & 15, lr = t >> 4;
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int64_t c0 = (int64_t)tc * kTile + 8 * l16;
  const T* x = reinterpret_cast<const T*>(p.x) + ((int64_t)tr * kTile + lr) * p.sr + c0 * p.sc;
  // rows and elements of this thread's part that exist
  const int64_t left_r = p.R - (int64_t)tr * kTile, left_c = p.C - c0;

  Vec8<DT> v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
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
  for (int i = 0; i < 8; i++) {
    if (!COLS && 16 * i >= left_r) break;  // few rows: nothing but latency
    if constexpr (ROWS) put_row<DT>(group_of(p.rows, (int64_t)tr * 8 + i, tc), v[i], lr, 8 * l16, lr + 16 * i < left_r);
    if constexpr (COLS) {
#pragma unroll
      for (int h = 0; h < DT::size / 2; h++)
        *reinterpret_cast<v4i*>(&tile[tile_word<W>(lr + 16 * i, l16 * 2 * DT::size + 4 * h)]) =
            v4i{(int)v[i].w[4 * h], (int)v[i].w[4 * h + 1], (int)v[i].w[4 * h + 2], (int)v[i].w[4 * h + 3]};
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    const int kb = (t & 63) >> 4, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int64_t left = p.C - (int64_t)tc * kTile;
    if constexpr (DT::size == 4) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int c = 16 * (4 * h + wave) + l16;
        u32 w[32];
#pragma unroll
        for (int r = 0; r < 32; r++) w[r] = tile[tile_word<W>(32 * kb + r, c)];
        put_col<DT>(group_of(p.cols, (int64_t)tc * 8 + 4 * h + wave, tr), w, l16, kb, c < left);
      }
    } else {
      pair_cols<DT, W>(tile, p.cols, (int64_t)tc * 8, tr, wave, l16, kb, kb, left);
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
  if (!(fabsf(f) < __builtin_inff()) || d == v) return (u >> 16) | ((u & 0xFFFFu) ? 1u : 0u);
  if (fabs(d) > fabs(v)) u -= 1;  // toward zero (f is not zero then)
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
  float tail = 0.f;
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
  const bool far = tail < -60.f;
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

// A tile of 32 NP rows of TW columns by 4 TW threads, each with eight elements of NP rows 32 apart.
// GRAD_PAIR: columns [c0, c0 + TW) of dh, g and u give a tile of dg and one of du. GRAD_GATE, GRAD_UP, GRAD_MIXED: a tile of
// d = [dg | du] at j0, all dg, all du, or some of either.
enum { GRAD_PAIR, GRAD_GATE, GRAD_UP, GRAD_MIXED };

template <class DT, int ACT, int MODE, int TW, int NP, bool ROWS, bool COLS>
__device__ __forceinline__ void grad_tile(const MxGradParams& p, u32* tile, int tr, int tc) {
  constexpr int LPR = TW / 8, TH = 32 * NP, TILE = TH * TW / 2;  // lanes per row, words of a tile
  typedef typename DT::T T;
  const int t = threadIdx.x, lc = t % LPR, lr = (t / LPR) & 15, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int half = wave / (LPR / 4);  // the 16-row half of a pass's 32 rows
  const int64_t F = p.F, left_r = p.M - (int64_t)tr * TH;
  const int64_t j = (int64_t)tc * TW + 8 * lc, c = MODE == GRAD_UP || (MODE == GRAD_MIXED && j >= F) ? j - F : j;
  const bool mixed = MODE == GRAD_MIXED && j < F && j + 8 > F;
  const int64_t row0 = (int64_t)tr * TH + 16 * half + lr;
  const T* dhp = reinterpret_cast<const T*>(p.dh) + row0 * p.ldh;
  const T* gp = reinterpret_cast<const T*>(p.gu) + row0 * p.ldgu;
  auto load = [&](int i) {
    GradIn<DT> x{zero8<DT>(), zero8<DT>(), zero8<DT>()};
    if (32 * i + 16 * half + lr >= left_r) return x;
    const T* dr = dhp + (int64_t)(32 * i) * p.ldh;
    const T* gr = gp + (int64_t)(32 * i) * p.ldgu;
    if (!mixed) {
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
    return x;
  };
  // places in a row of the row tensor: the tile's, and du's (F is a multiple of 32, not of a stage)
  const int64_t up_at = F + (int64_t)tc * TW;
  const int stage = tc / (kTile / TW), pos = (tc % (kTile / TW)) * TW + 8 * lc;
  const int up_stage = (int)(up_at / kTile), up_pos = (int)(up_at % kTile) + 8 * lc;
  GradIn<DT> next = load(0);
#pragma unroll 1
  for (int i = 0; i < NP; i++) {
    const GradIn<DT> x = next;
    if (i + 1 < NP) next = load(i + 1);
    const int in = 32 * i + 16 * half;  // the 16-row group's first row in the tile
    Vec8<MxBF16> d = zero8<MxBF16>(), du = zero8<MxBF16>();
    if (in < left_r) {
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
      if constexpr (ROWS) {
        const int64_t group = (int64_t)tr * (2 * NP) + 2 * i + half;
        const bool live = in + lr < left_r && (MODE != GRAD_PAIR || c < F);
        put_row<MxBF16>(group_of(p.rows, group, stage), d, lr, pos, live);
        if constexpr (MODE == GRAD_PAIR) put_row<MxBF16>(group_of(p.rows, group, up_stage), du, lr, up_pos, live);
      }
    }
    if constexpr (COLS) {
      const int at = tile_word<TW / 2>(in + lr, 4 * lc);
      *reinterpret_cast<v4i*>(&tile[at]) = v4i{(int)d.w[0], (int)d.w[1], (int)d.w[2], (int)d.w[3]};
      if constexpr (MODE == GRAD_PAIR) *reinterpret_cast<v4i*>(&tile[TILE + at]) = v4i{(int)du.w[0], (int)du.w[1], (int)du.w[2], (int)du.w[3]};
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    const int64_t col0 = (int64_t)tc * TW;
    const int stage_c = tr / (kTile / TH), kb0 = tr % (kTile / TH) * NP;
    const int l16 = t & 15;
    // sixteen lanes take 16 pairs of columns of one block of 32 rows
    int s16 = t >> 4;
    const int kb = s16 % NP, w = s16 / NP % (TW / 32), side = s16 / NP / (TW / 32);
    if (side < (MODE == GRAD_PAIR ? 2 : 1))
      pair_cols<MxBF16, TW / 2>(tile + side * TILE, p.cols, (col0 + (side ? F : 0)) / 16, stage_c, w, l16, kb, kb0 + kb,
                                (MODE == GRAD_PAIR ? F : 2 * F) - col0);
  }
}

// F a multiple of 32, so that blocks along d = [dg | du] belong to one side: every input is read once.
// Two blocks of 512 threads (or four of 256) per compute unit, 128 registers, where that spills next to nothing; float32
// inputs and erf take more.
template <class DT, int ACT, int TW, int NP, bool ROWS, bool COLS>
__global__ __launch_bounds__(4 * TW, DT::size == 4 || ACT == SVDQ_ACT_GELU ? 2 : 4) void k_mx_gated_grad(MxGradParams p, int tiles_c) {
  __shared__ __align__(16) u32 tile[COLS ? 32 * NP * TW : 4];
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  grad_tile<DT, ACT, GRAD_PAIR, TW, NP, ROWS, COLS>(p, tile, tr, tc);
  if constexpr (ROWS) {
    // the row tensor's padding past 2 F, zero codes and bytes, by the last column of blocks
    if (tc == tiles_c - 1) {
      const int l16 = threadIdx.x & 15, lr = threadIdx.x >> 4;
      for (int st = (int)(2 * p.F / kTile); st < p.rows.kq; st++) {
        const bool past = (int64_t)st * kTile + 8 * l16 >= 2 * p.F;
        for (int r = lr; r < 32 * NP; r += TW / 4) {
          const int64_t row = (int64_t)tr * (32 * NP) + r;
          put_row<MxBF16>(group_of(p.rows, row >> 4, st), zero8<MxBF16>(), row & 15, 8 * l16, past && row < p.M);
        }
      }
    }
  }
}

// Any F: tiles of d itself. The two that read the same dh and g, one on either side of F, go to blocks 8 apart:
// neighbours on one XCD, so that the second finds them in its L2.
template <class DT, int ACT, int TW, int NP, bool ROWS, bool COLS>
__global__ __launch_bounds__(4 * TW, DT::size == 4 || ACT == SVDQ_ACT_GELU ? 2 : 4) void k_mx_gated_grad_any(MxGradParams p, int tiles_c, int pairs) {
  __shared__ __align__(16) u32 tile[COLS ? 16 * NP * TW : 4];
  const int64_t id = (int64_t)(blockIdx.x >> 4) * 8 + (blockIdx.x & 7);
  const int tr = (int)(id / pairs), pair = (int)(id - (int64_t)tr * pairs), side = (blockIdx.x >> 3) & 1;
  const int first_up = (int)(p.F / TW), tc = side ? first_up + pair : pair;
  if (side ? tc >= tiles_c : tc >= first_up) return;
  if (COLS ? tr >= p.cols.kq * (4 / NP) : (int64_t)tr * (32 * NP) >= p.M) return;
  if (side == 0)
    grad_tile<DT, ACT, GRAD_GATE, TW, NP, ROWS, COLS>(p, tile, tr, tc);
  else if (pair != 0)
    grad_tile<DT, ACT, GRAD_UP, TW, NP, ROWS, COLS>(p, tile, tr, tc);
  else
    grad_tile<DT, ACT, GRAD_MIXED, TW, NP, ROWS, COLS>(p, tile, tr, tc);
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

hipError_t launch_mx_quantize(const MxQuantParams& p0, int dtype, hipStream_t stream) {
  MxQuantParams p = p0;
  if (p.sc != 1 && p.sr == 1) {  // columns are contiguous: the transpose's rows
    const MxQuantParams q = p;
    p.R = q.C, p.C = q.R, p.sr = q.sc, p.sc = q.sr, p.rows = q.cols, p.cols = q.rows;
  }
  // a direction that is written covers its padding too
  const int64_t tc = p.rows.codes ? p.rows.kq : tiles_of(p.C), tr = p.cols.codes ? p.cols.kq : tiles_of(p.R);
  if (tc * tr > 0x7FFFFFFF) return hipErrorInvalidValue;
  return with_dtype(dtype, [&](auto d) {
    typedef decltype(d) DT;
    const dim3 grid((unsigned)(tc * tr));
    if (p.rows.codes && p.cols.codes)
      k_mx_quantize<DT, true, true><<<grid, 256, 0, stream>>>(p, (int)tc);
    else if (p.rows.codes)
      k_mx_quantize<DT, true, false><<<grid, 256, 0, stream>>>(p, (int)tc);
    else
      k_mx_quantize<DT, false, true><<<grid, 256, 0, stream>>>(p, (int)tc);
    return hipGetLastError();
  });
}

hipError_t launch_mx_dequantize(const MxDequantParams& p, int dtype, hipStream_t stream) {
  const int64_t st = tiles_of(p.K), blocks = (p.rows + 63) / 64 * st;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  return with_dtype(dtype, [&](auto d) {
    k_mx_dequantize<decltype(d)><<<dim3((unsigned)blocks), 256, 0, stream>>>(p, (int)st);
    return hipGetLastError();
  });
}

template <class DT, int ACT, int NP, bool ROWS, bool COLS>
static hipError_t launch_grad_t(const MxGradParams& p, hipStream_t stream) {
  constexpr int TW = kGradCols, TH = 32 * NP;
  const int64_t tr = COLS ? (int64_t)p.cols.kq * (kTile / TH) : (p.M + TH - 1) / TH;
  // Measured at 4096 rows, bf16, silu, both directions: @@PAIR@@ us for F = 12288 as pairs, @@ANY@@ us for F = 12300.
  if (p.F % kMxBlock == 0) {
    const int64_t tc = (p.F + TW - 1) / TW;
    if (tc * tr > 0x7FFFFFFF) return hipErrorInvalidValue;
    k_mx_gated_grad<DT, ACT, TW, NP, ROWS, COLS><<<dim3((unsigned)(tc * tr)), 4 * TW, 0, stream>>>(p, (int)tc);
    return hipGetLastError();
  }
  // tiles of [0, 2F), with the row tensor's padding; those that begin below F, and those from the one that holds F on
  const int64_t tc = ROWS ? (int64_t)p.rows.kq * (kTile / TW) : (2 * p.F + TW - 1) / TW;
  const int64_t below = p.F / TW, pairs = tc - below > below ? tc - below : below;
  const int64_t blocks = (pairs * tr + 7) / 8 * 16;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  k_mx_gated_grad_any<DT, ACT, TW, NP, ROWS, COLS><<<dim3((unsigned)blocks), 4 * TW, 0, stream>>>(p, (int)tc, (int)pairs);
  return hipGetLastError();
}

template <class DT, int ACT, int NP>
static hipError_t launch_grad_np(const MxGradParams& p, hipStream_t stream) {
  if (p.rows.codes && p.cols.codes) return launch_grad_t<DT, ACT, NP, true, true>(p, stream);
  return p.rows.codes ? launch_grad_t<DT, ACT, NP, true, false>(p, stream) : launch_grad_t<DT, ACT, NP, false, true>(p, stream);
}

// Tiles of 128 rows fill whole 64-byte rows of the transpose's codes; where they would leave the chip with less than
// @@NB@@ blocks per compute unit, tiles of 32 rows, whose loads all wait at once.
template <class DT, int ACT>
static hipError_t launch_grad_act(const MxGradParams& p, hipStream_t stream) {
  const int64_t blocks = tiles_of(p.M) * ((p.F + kGradCols - 1) / kGradCols);
  return blocks < kGradFew ? launch_grad_np<DT, ACT, 1>(p, stream) : launch_grad_np<DT, ACT, 4>(p, stream);
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
