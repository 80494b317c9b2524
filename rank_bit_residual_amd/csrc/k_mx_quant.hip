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

constexpr int kTile = 128;

__device__ inline u32 quad_max(u32 v) {
  v = max(v, (u32)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // quad_perm [1,0,3,2]
  v = max(v, (u32)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // quad_perm [2,3,0,1]
  return v;
}

// Quantises a row's eight elements per lane: lanes 4 j .. 4 j + 3 hold block j of the row's stage,
// sixteen lanes a stage. Writes the codes, and the four scale bytes as one word.
template <class DT>
__device__ inline void put_row(const MxOut& o, const Vec8<DT>& v, int64_t row, int stage, int lane16, bool live) {
  const u32 byte = mx_scale_byte(quad_max(amax_bits<DT>(v.w)));
  const u32 word = codes8<DT>(v.w, byte);
  u32 s = byte << (8 * (lane16 >> 2));
  s |= (u32)__shfl_xor((int)s, 4, 64);
  s |= (u32)__shfl_xor((int)s, 8, 64);
  if (!live) return;
  uint8_t* tile = o.codes + (((row >> 4) * o.kq + stage) << 10) + ((row & 15) << 6);
  *reinterpret_cast<u32*>(tile + lane16 * 4) = word;
  if (lane16 == 0) *reinterpret_cast<u32*>(o.scales + mx_scale_tiled_index(row, 4 * stage, o.kq)) = s;
}

// Quantises a column's 32 elements (one block of the transpose) held by a lane: N words of pairs
// or values. kb: the block's place in its stage, held by lanes 16 kb .. 16 kb + 15.
template <class DT, int N>
__device__ inline void put_col(const MxOut& o, const u32 (&w)[N], int64_t col, int stage, int kb, bool live) {
  const u32 byte = mx_scale_byte(amax_bits<DT>(w));
  v4i c;
#pragma unroll
  for (int q = 0; q < 4; q++) c[q] = (int)codes8<DT>(w + N / 4 * q, byte);
  u32 s = byte << (8 * kb);
  s |= (u32)__shfl_xor((int)s, 16, 64);
  s |= (u32)__shfl_xor((int)s, 32, 64);
  if (!live) return;
  uint8_t* tile = o.codes + (((col >> 4) * o.kq + stage) << 10) + ((col & 15) << 6);
  *reinterpret_cast<v4i*>(tile + kb * 16) = c;
  if (kb == 0) *reinterpret_cast<u32*>(o.scales + mx_scale_tiled_index(col, 4 * stage, o.kq)) = s;
}

// LDS copy of a tile: W words per row. A column reader's lanes are 16 columns x 4 blocks of 32
// rows; moving a row's 16-word groups by its block's number puts the four blocks on different banks.
template <int W>
__device__ inline int tile_word(int row, int word) {
  return row * W + (word ^ (((row >> 5) & 3) << 4));
}

// ------------------------------------------------------------------------------ quantise
// Block: 256 threads; thread t holds elements [8 (t % 16), + 8) of rows t / 16 + 16 i.
template <class DT, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void k_mx_quantize(MxQuantParams p, int tiles_c) {
  constexpr int W = kTile * DT::size / 4;  // words per tile row
  __shared__ __align__(16) u32 tile[COLS ? kTile * W : 4];
  typedef typename DT::T T;
  const T* x = reinterpret_cast<const T*>(p.x);
  const int t = threadIdx.x, l16 = t & 15;
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int64_t r0 = (int64_t)tr * kTile + (t >> 4), c0 = (int64_t)tc * kTile + 8 * l16;

  Vec8<DT> v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int64_t r = r0 + 16 * i;
    if (r >= p.R) {
      v[i] = zero8<DT>();
    } else if (p.sc == 1) {
      v[i] = load8<DT>(x + r * p.sr, c0, p.C);
    } else {
      v[i] = zero8<DT>();
#pragma unroll
      for (int q = 0; q < 8; q++) {
        if (c0 + q >= p.C) continue;
        const T e = x[r * p.sr + (c0 + q) * p.sc];
        if constexpr (DT::size == 4)
          v[i].w[q] = __float_as_uint(e);
        else
          v[i].w[q >> 1] |= (u32)e << (16 * (q & 1));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int64_t r = r0 + 16 * i;
    if constexpr (ROWS) put_row<DT>(p.rows, v[i], r, tc, l16, r < p.R);
    if constexpr (COLS) {
      const int lr = (t >> 4) + 16 * i;
#pragma unroll
      for (int h = 0; h < DT::size / 2; h++)
        *reinterpret_cast<v4i*>(&tile[tile_word<W>(lr, l16 * 2 * DT::size + 4 * h)]) =
            v4i{(int)v[i].w[4 * h], (int)v[i].w[4 * h + 1], (int)v[i].w[4 * h + 2], (int)v[i].w[4 * h + 3]};
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    const int kb = (t & 63) >> 4, wave = t >> 6;
    if constexpr (DT::size == 4) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int c = 64 * h + 16 * wave + l16;
        u32 w[32];
#pragma unroll
        for (int r = 0; r < 32; r++) w[r] = tile[tile_word<W>(32 * kb + r, c)];
        const int64_t col = (int64_t)tc * kTile + c;
        put_col<DT>(p.cols, w, col, tr, kb, col < p.C);
      }
    } else {
      // a lane takes a pair of columns: the low halves of its words, then the high halves
      const int pr = 16 * wave + l16;
      u32 lo[16], hi[16];
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const u32 a = tile[tile_word<W>(32 * kb + 2 * r, pr)], b = tile[tile_word<W>(32 * kb + 2 * r + 1, pr)];
        lo[r] = __builtin_amdgcn_perm(b, a, 0x05040100u);
        hi[r] = __builtin_amdgcn_perm(b, a, 0x07060302u);
      }
      const int64_t col = (int64_t)tc * kTile + 2 * pr;
      put_col<DT>(p.cols, lo, col, tr, kb, col < p.C);
      put_col<DT>(p.cols, hi, col + 1, tr, kb, col + 1 < p.C);
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
// and |v| + err agree in the bits above those; an unsettled v (about one in 20000 for pre-activations
// of unit scale) is computed in binary64 and kept as a float32 that lies on the same side of every border:
// truncated, with the lowest bit set if anything was cut off.
__device__ inline bool unsettled(float v, float err) {
  const float a = fabsf(v);
  return (__float_as_uint(a - err) >> 21) != (__float_as_uint(a + err) >> 21);
}

__device__ inline float to_odd(double v) {
  const float f = (float)v;
  if (!(fabsf(f) < __builtin_inff())) return f;  // NaN, or too large: the block reads as NaN
  const double d = (double)f;
  if (d == v) return f;
  u32 u = __float_as_uint(f);
  if (fabs(d) > fabs(v)) u -= 1;  // toward zero (f is not zero then)
  if (u << 1 == 0) u |= v < 0 ? 0x80000000u : 0u;
  return __uint_as_float(u | 1u);
}

template <int ACT>
__device__ inline float grad_exact(bool up, float dh, float g, float u) {
  const ActValue<double> r = act_value<ACT, double>((double)g);
  return to_odd(up ? (double)dh * r.a : ((double)dh * (double)u) * r.d);
}

// One side of eight elements: dg (up = false) or du.
template <int ACT>
__device__ inline u32 grad8(bool up, const float* dh, const float* g, const float* u, float* v) {
  u32 open = 0;
#pragma unroll
  for (int q = 0; q < 8; q++) {
    const ActValue<float> r = act_value<ACT, float>(g[q]);
    float err;
    if (up) {
      v[q] = dh[q] * r.a;
      err = fabsf(v[q]) * r.rel_a;
    } else {
      const float a = dh[q] * u[q];
      v[q] = a * r.d;
      err = fabsf(a) * r.abs_d;
    }
    // near the ends of the float32 range products lose digits that the bounds do not count (relu's
    // zeros are exact)
    const float size = fabsf(v[q]);
    const bool ends = !(size < 0x1p126f) || (size < 0x1p-100f && (ACT == SVDQ_ACT_RELU ? v[q] : dh[q]) != 0.f);
    open |= unsettled(v[q], err) || ends ? 1u << q : 0u;
  }
  return open;
}

template <class DT>
__device__ inline float pick(const Vec8<DT>& v, int q) {
  u32 w = v.w[0];
#pragma unroll
  for (int i = 1; i < DT::size * 2; i++) w = (DT::size == 4 ? q : q >> 1) == i ? v.w[i] : w;
  if constexpr (DT::size == 4)
    return __uint_as_float(w);
  else
    return DT::load((uint16_t)(w >> (16 * (q & 1))));
}

// Block: 512 threads, a 128 x 128 tile of d = [dg | du]; thread t holds elements [8 (t % 16), + 8)
// of rows t / 16 + 32 i.
template <class DT, int ACT, bool ROWS, bool COLS>
__global__ __launch_bounds__(512) void k_mx_gated_grad(MxGradParams p, int tiles_c) {
  __shared__ __align__(16) u32 tile[COLS ? kTile * kTile : 4];
  typedef typename DT::T T;
  const T* dhp = reinterpret_cast<const T*>(p.dh);
  const T* gup = reinterpret_cast<const T*>(p.gu);
  const int t = threadIdx.x, l16 = t & 15;
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int64_t j0 = (int64_t)tc * kTile + 8 * l16;  // place in [0, 2F)
  const int64_t F = p.F;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int lr = (t >> 4) + 32 * i;
    const int64_t r = (int64_t)tr * kTile + lr;
    Vec8<MxF32> o = zero8<MxF32>();
    if (r < p.M && j0 < 2 * F) {
      Vec8<DT> dh = zero8<DT>(), g = zero8<DT>(), u = zero8<DT>();
      const T* dr = dhp + r * p.ldh;
      const T* gr = gup + r * p.ldgu;
      // this lane's elements: gate columns [j0, F), then up columns [max(j0, F) - F, 2F)
      u32 ups = 0;  // bit q: element q belongs to du
      if (j0 + 8 <= F || j0 >= F) {
        const bool up = j0 >= F;
        const int64_t c = up ? j0 - F : j0;
        dh = load8<DT>(dr, c, F);
        g = load8<DT>(gr, c, F);
        if (!up) u = load8<DT>(gr + F, c, F);
        ups = up ? 0xFFu : 0u;
      } else {
#pragma unroll
        for (int q = 0; q < 8; q++) {
          const int64_t j = j0 + q;
          if (j >= 2 * F) continue;
          const int64_t c = j < F ? j : j - F;
          if constexpr (DT::size == 4) {
            dh.w[q] = __float_as_uint(dr[c]);
            g.w[q] = __float_as_uint(gr[c]);
            u.w[q] = __float_as_uint(gr[F + c]);
          } else {
            dh.w[q >> 1] |= (u32)dr[c] << (16 * (q & 1));
            g.w[q >> 1] |= (u32)gr[c] << (16 * (q & 1));
            u.w[q >> 1] |= (u32)gr[F + c] << (16 * (q & 1));
          }
          ups |= j < F ? 0u : 1u << q;
        }
      }
      float dv[8], gv[8], uv[8], v[8];
#pragma unroll
      for (int q = 0; q < 8; q++) {
        dv[q] = elem<DT>(dh, q);
        gv[q] = elem<DT>(g, q);
        uv[q] = elem<DT>(u, q);
      }
      u32 open = 0;
      if (ups != 0xFFu) {
        open = grad8<ACT>(false, dv, gv, uv, v) & ~ups;
#pragma unroll
        for (int q = 0; q < 8; q++) o.w[q] = __float_as_uint(v[q]);
      }
      if (ups) {
        open |= grad8<ACT>(true, dv, gv, uv, v) & ups;
#pragma unroll
        for (int q = 0; q < 8; q++) o.w[q] = (ups >> q & 1) ? __float_as_uint(v[q]) : o.w[q];
      }
      while (open) {
        const int q = __builtin_ctz(open);
        open &= open - 1;
        const u32 e = __float_as_uint(grad_exact<ACT>(ups >> q & 1, pick<DT>(dh, q), pick<DT>(g, q), pick<DT>(u, q)));
#pragma unroll
        for (int k = 0; k < 8; k++) o.w[k] = k == q ? e : o.w[k];
      }
      // elements past 2F came from zeros: dh = 0 gives 0, unless the activation of 0 is not finite
    }
    if constexpr (ROWS) put_row<MxF32>(p.rows, o, r, tc, l16, r < p.M);
    if constexpr (COLS) {
#pragma unroll
      for (int h = 0; h < 2; h++)
        *reinterpret_cast<v4i*>(&tile[tile_word<kTile>(lr, 8 * l16 + 4 * h)]) =
            v4i{(int)o.w[4 * h], (int)o.w[4 * h + 1], (int)o.w[4 * h + 2], (int)o.w[4 * h + 3]};
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    const int kb = (t & 63) >> 4, c = 16 * (t >> 6) + l16;
    u32 w[32];
#pragma unroll
    for (int r = 0; r < 32; r++) w[r] = tile[tile_word<kTile>(32 * kb + r, c)];
    const int64_t col = (int64_t)tc * kTile + c;
    put_col<MxF32>(p.cols, w, col, tr, kb, col < 2 * F);
  }
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

template <class DT, int ACT>
static hipError_t launch_grad_t(const MxGradParams& p, hipStream_t stream) {
  const int64_t tc = p.rows.codes ? p.rows.kq : tiles_of(2 * p.F), tr = p.cols.codes ? p.cols.kq : tiles_of(p.M);
  if (tc * tr > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 grid((unsigned)(tc * tr));
  if (p.rows.codes && p.cols.codes)
    k_mx_gated_grad<DT, ACT, true, true><<<grid, 512, 0, stream>>>(p, (int)tc);
  else if (p.rows.codes)
    k_mx_gated_grad<DT, ACT, true, false><<<grid, 512, 0, stream>>>(p, (int)tc);
  else
    k_mx_gated_grad<DT, ACT, false, true><<<grid, 512, 0, stream>>>(p, (int)tc);
  return hipGetLastError();
}

hipError_t launch_mx_gated_grad(const MxGradParams& p, int dtype, hipStream_t stream) {
  return with_dtype(dtype, [&](auto d) {
    typedef decltype(d) DT;
    switch (p.act) {
      case SVDQ_ACT_SILU: return launch_grad_t<DT, SVDQ_ACT_SILU>(p, stream);
      case SVDQ_ACT_GELU: return launch_grad_t<DT, SVDQ_ACT_GELU>(p, stream);
      case SVDQ_ACT_GELU_TANH: return launch_grad_t<DT, SVDQ_ACT_GELU_TANH>(p, stream);
      default: return launch_grad_t<DT, SVDQ_ACT_RELU>(p, stream);
    }
  });
}

}  // namespace svdq
