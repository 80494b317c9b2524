// Layer norm on gfx950: y = (x - mean) / sqrt(var + eps) * weight + bias of each row, as it is or as the 8-bit or MXFP4 tensor of y,
// and its backward pass.
//
// Forward: a row is read once and stays in the registers of the threads that share it. Sums and y are binary64, whose sums and
// products issue nearly as fast as float32's where waves share a SIMD (with eight, 2.0 to 2.2 ns an instruction against 1.8; conversions to
// it take 3.6): with d = x - x[0], mean = x[0] + sum d / K and var = sum d^2 / K - (sum d / K)^2 come from one reduction, and since
// (x[0] - mean)^2 <= K var the subtraction costs log2 K of 53 bits at most. y is rounded to
// float32 once, and that is what is quantised or rounded on to the output's type; a code is decided by comparing with a border, so
// rounding earlier would move one now and then. Memory bounds float32 rows and large 16-bit ones (8192 x 8192 98 us and 53, 5.5 and 5.1
// TB/s); where fewer bytes leave, the binary64 steps (12 an element, four of them conversions to it) and the codes do: to 8 bits 69 us, to MXFP4 52,
// of 38 and 32 for the bytes alone. The parameters wait as float32, as binary64 they would cost the third wave of registers.
//
// Backward: with xh = (x - mean) rstd and g = dy weight, dx = rstd (g - mean(g) - xh mean(g xh)): one reduction, with dy and x in
// registers. A thread keeps the same columns in every row of its block, so dweight = sum dy xh and dbias = sum dy are running sums
// in registers, over 1024 rows at most; each block leaves its own, and a last kernel adds them in binary64 in the blocks' order. Memory
// bounds it: 8192 x 8192 bf16 75 us (5.4 TB/s) and 5 for the last kernel.
#include <type_traits>

#include "i8.h"
#include "i8_device.h"
#include "mx_rows.h"

namespace svdq {
namespace dev {

enum { NORM_Y, NORM_I8, NORM_MX };

// Elements [c, c + 8) of a parameter vector of K, or `none` without one; zeros past its end.
template <class DT>
__device__ inline void param8(float (&w)[8], const void* src, bool f32, int64_t c, int64_t K, float none) {
  if (!src) {
#pragma unroll
    for (int k = 0; k < 8; k++) w[k] = none;
  } else if (f32) {
    const Vec8<MxF32> v = load8<MxF32>(reinterpret_cast<const float*>(src), c, K);
#pragma unroll
    for (int k = 0; k < 8; k++) w[k] = elem<MxF32>(v, k);
  } else {
    const Vec8<DT> v = load8<DT>(reinterpret_cast<const typename DT::T*>(src), c, K);
#pragma unroll
    for (int k = 0; k < 8; k++) w[k] = elem<DT>(v, k);
  }
}

// ------------------------------------------------------------------------------ forward
struct RowStats {
  double mean, rstd;
};

// 1 / sqrt(v), to 2^-51: the hardware's estimate is off by less than 2^-22, and one step of third order cubes that.
__device__ inline double rsqrt64(double v) {
  if (!(v >= 0x1p-1000)) return 1.0 / sqrt(v);  // near or at zero, or NaN
  const double r = __builtin_amdgcn_rsq(v), e = __builtin_fma(-(v * r), r, 1.0);
  return __builtin_fma(r * e, __builtin_fma(0.375, e, 0.5), r);
}

// A row's first element, as bits and as a value.
template <class DT>
__device__ inline u32 first_bits(const typename DT::T* x) {
  if constexpr (DT::size == 4)
    return __float_as_uint(x[0]);
  else
    return x[0];
}
template <class DT>
__device__ inline double bits_value(u32 bits) {
  if constexpr (DT::size == 4)
    return __uint_as_float(bits);
  else
    return DT::load((uint16_t)bits);
}

// This thread's share of sum d and sum d^2.
template <class DT>
__device__ inline void add_stats(const Vec8<DT>& v, double pivot, Sums2& sum, int64_t n = 8) {
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const double d = k < n ? (double)elem<DT>(v, k) - pivot : 0.0;
    sum.a += d;
    sum.b = __builtin_fma(d, d, sum.b);
  }
}

// Keeps the elements in their own type, so that their float64 values do not live on in registers.
template <class DT>
__device__ __forceinline__ void settle(Vec8<DT>& v) {
#pragma unroll
  for (int k = 0; k < DT::size * 2; k++) asm volatile("" : "+v"(v.w[k]));
}

// Eight columns' weight and bias.
struct Params8 {
  float w[8], b[8];
};
template <class DT>
__device__ inline void load_params(Params8& q, const NormParams& p, int64_t c) {
  param8<DT>(q.w, p.weight, p.param_f32, c, p.K, 1.f);
  param8<DT>(q.b, p.bias, p.param_f32, c, p.K, 0.f);
}

// y of eight elements, as float32; zeros past the row's end.
template <class DT>
__device__ inline void norm8(float (&y)[8], const Vec8<DT>& v, int64_t c, int64_t K, const Params8& q, const RowStats& st) {
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const double xh = ((double)elem<DT>(v, k) - st.mean) * st.rstd;
    y[k] = (float)__builtin_fma(xh, (double)q.w[k], (double)q.b[k]);
  }
  if (c + 8 > K) {
#pragma unroll
    for (int k = 0; k < 8; k++) y[k] = c + k < K ? y[k] : 0.f;
  }
}

__device__ __forceinline__ void settle(Params8& q) {
#pragma unroll
  for (int k = 0; k < 8; k++) asm volatile("" : "+v"(q.w[k]), "+v"(q.b[k]));
}

__device__ inline u32 amax8(const float (&y)[8]) {
  u32 m = 0;
#pragma unroll
  for (int k = 0; k < 8; k++) m = max(m, __float_as_uint(y[k]) & 0x7FFFFFFFu);
  return m;
}

template <class DT, int OUT>
__device__ inline void put8(const NormParams& p, int64_t row, int64_t c, const float (&y)[8], const Scale8& q) {
  if constexpr (OUT == NORM_Y) {
    if (c < p.K) store8<DT>(reinterpret_cast<typename DT::T*>(p.y) + row * p.ldy, c, p.K, y);
  } else if constexpr (OUT == NORM_I8) {
    if (c < (int64_t)p.i8.kq * 64) *reinterpret_cast<v2u*>(p.i8.codes + i8_at(row, c, p.i8.kq)) = codes8x8(y, q);
  } else {
    Vec8<MxF32> v;
#pragma unroll
    for (int k = 0; k < 8; k++) v.w[k] = __float_as_uint(y[k]);
    const int64_t stage = c >> 7;
    put_row<MxF32>(group_of(p.mx, row >> 4, stage), v, (u32)(row & 15), (u32)(c & 127), c < (int64_t)p.mx.kq * 128);
  }
}

// T threads share a row of eight elements or more and hold NV times eight each; NV = 0: a row of any length, read once for its statistics and
// again for y (twice for 8-bit codes). A block takes rows one after another: its columns' parameters stay in registers, and
// the next row is on its way while one is worked on.
template <class DT, int T, int NV, int OUT>
__global__ __launch_bounds__(T < 256 ? 256 : T, NV == 2 ? 4 : 1) void k_norm(NormParams p) {
  typedef typename DT::T E;
  constexpr int RPB = T < 256 ? 256 / T : 1, WAVES = T / 64, N = NV ? NV : 1;
  __shared__ Sums2 red[2][RPB][4 * WAVES];
  __shared__ u32 redm[2][RPB][4 * WAVES];
  const int t = threadIdx.x % T, sub = threadIdx.x / T;
  // threads past the end of a row take part up to the end of the codes' padding
  const int64_t Kp = OUT == NORM_Y ? p.K : (OUT == NORM_I8 ? (int64_t)p.i8.kq * 64 : (int64_t)p.mx.kq * 128);
  auto at = [&](int j) { return (int64_t)(j * T + t) * 8; };
  auto load = [&](Vec8<DT>(&v)[N], u32& pivot, int64_t row) {
    const E* x = reinterpret_cast<const E*>(p.x) + row * p.ldx;
    pivot = first_bits<DT>(x);
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; j++) v[j] = load8_last<DT>(x, at(j), p.K);
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  const double k1 = 1.0 / (double)p.K;
  Vec8<DT> v[N], next[N];
  u32 pivot_bits = 0, pivot_next = 0;
  // rows of a block: its threads stay together (they share barriers), so past the last row some repeat it
  int64_t first = (int64_t)blockIdx.x * RPB;
  load(v, pivot_bits, min(first + sub, p.M - 1));
  Params8 q[N];
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; j++) load_params<DT>(q[j], p, at(j));
  }
  int flip = 0;
  for (; first < p.M; first += step, flip ^= 1) {
    const int64_t row = min(first + sub, p.M - 1);
    if (first + step < p.M) load(next, pivot_next, min(first + step + sub, p.M - 1));
    const E* x = reinterpret_cast<const E*>(p.x) + row * p.ldx;
    const double pivot = bits_value<DT>(pivot_bits);
    Sums2 sum{0, 0};
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; j++) {
        fit8<DT>(v[j], at(j), p.K, pivot_bits);  // past the row's end its first element: it adds nothing to the differences
        add_stats<DT>(v[j], pivot, sum);
        settle(v[j]);
        settle(q[j]);
      }
    } else {
      for (int64_t c = (int64_t)t * 8; c < p.K; c += T * 8) add_stats<DT>(load8<DT>(x, c, p.K), pivot, sum, p.K - c);
    }
    if constexpr (WAVES > 1) {
      sum = row_join(sum, add2);
      // two buffers: a wave may reach the next row's write while others still read this one's
      if ((t & 15) == 0) red[flip][sub][t >> 4] = sum;
      lds_barrier();
      sum = waves_join<WAVES>(red[flip][sub], add2);
    } else {
      sum = wave_join(sum, add2);
    }
    const double ds = sum.a * k1;
    double var = __builtin_fma(sum.b, k1, -ds * ds);
    var = var < 0 ? 0 : var;  // NaN stays
    const RowStats st{pivot + ds, rsqrt64(var + p.eps)};
    if (t == 0 && p.mean) p.mean[row] = (float)st.mean, p.rstd[row] = (float)st.rstd;

    Scale8 scale{0.f, 0.f};
    float y[N][8];
    if constexpr (OUT == NORM_I8) {
      u32 most = 0;
      if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; j++) {
          norm8<DT>(y[j], v[j], at(j), p.K, q[j], st);
          most = max(most, amax8(y[j]));
        }
      } else {
        for (int64_t c = (int64_t)t * 8; c < p.K; c += T * 8) {
          load_params<DT>(q[0], p, c);
          norm8<DT>(y[0], load8<DT>(x, c, p.K), c, p.K, q[0], st);
          most = max(most, amax8(y[0]));
        }
      }
      if constexpr (WAVES > 1) {
        most = row_join(most, umax2);
        if ((t & 15) == 0) redm[flip][sub][t >> 4] = most;
        lds_barrier();
        most = waves_join<WAVES>(redm[flip][sub], umax2);
      } else {
        most = wave_umax(most);
      }
      scale = scale8(most);
      if (t == 0) p.i8.scales[row] = scale.s;
    }
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; j++) {
        if constexpr (OUT != NORM_I8) norm8<DT>(y[j], v[j], at(j), p.K, q[j], st);
        put8<DT, OUT>(p, row, at(j), y[j], scale);
        v[j] = next[j];
      }
    } else {
      // whole waves: an MXFP4 block's four lanes agree on its maximum
      for (int64_t c0 = (int64_t)(t & ~63) * 8; c0 < Kp; c0 += T * 8) {
        const int64_t c = c0 + 8 * (t & 63);
        load_params<DT>(q[0], p, c);
        norm8<DT>(y[0], load8<DT>(x, c, p.K), c, p.K, q[0], st);
        put8<DT, OUT>(p, row, c, y[0], scale);
      }
    }
    pivot_bits = pivot_next;
  }
}

// ------------------------------------------------------------------------------ backward
template <class DT>
struct GradRow {
  Vec8<DT> dy, x;
};

// T threads share a row of eight elements or more, NV times eight columns each, the same ones in every row that the block takes; only the last
// of a thread's vectors may pass the row's end (K > 8 T (NV - 1)). AHEAD: the
// next row is requested before this one is worked on; with four vectors a thread it has no room (4096 x 16384 bf16 97 us without, 108
// with, float32 179 and 243; two vectors of 1024 threads, which have half the registers, 130 and 286).
template <class DT, int T, int NV, bool AHEAD>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_norm_grad(NormGradParams p, float* part) {
  typedef typename DT::T E;
  constexpr int RPB = T < 256 ? 256 / T : 1, WAVES = T / 64;
  __shared__ float red[2][2][WAVES];
  __shared__ float wide[RPB > 1 ? RPB * NV * 16 * T : 1];
  const int t = threadIdx.x % T, sub = threadIdx.x / T, wave = t >> 6;
  float w[NV][8], dw[NV][8] = {}, db[NV][8] = {};
#pragma unroll
  for (int j = 0; j < NV; j++) param8<DT>(w[j], p.weight, p.param_f32, (int64_t)(j * T + t) * 8, p.K, 1.f);
  const float k1 = 1.f / (float)p.K;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + sub;
  GradRow<DT> cur[NV];
  float mean = 0.f, rstd = 0.f;
  auto load = [&](GradRow<DT>(&to)[NV], int64_t r, float& mu, float& rs) {
    if (r >= p.M) return;
    mu = p.mean[r], rs = p.rstd[r];
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const int64_t c = (int64_t)(j * T + t) * 8;
      to[j].dy = load8_last<DT>(reinterpret_cast<const E*>(p.dy) + r * p.lddy, c, p.K);
      to[j].x = load8_last<DT>(reinterpret_cast<const E*>(p.x) + r * p.ldx, c, p.K);
    }
  };
  load(cur, row, mean, rstd);
  int flip = 0;
  for (; row < p.M; row += step, flip ^= 1) {
    GradRow<DT> next[AHEAD ? NV : 1];
    float mu = 0.f, rs = 0.f;
    if constexpr (AHEAD) load(next, row + step, mu, rs);
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; j++) {
      if (j == NV - 1) {
        fit8<DT>(cur[j].dy, (int64_t)(j * T + t) * 8, p.K);
        turn8<DT>(cur[j].x, (int64_t)(j * T + t) * 8, p.K);  // not zeros: (0 - mean) rstd may be infinite, and 0 times it NaN
        if constexpr (!AHEAD) {  // or float32 rows of 16384 spill twice as much, 188 us and not 177
          settle(cur[j].dy);
          settle(cur[j].x);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float dy = elem<DT>(cur[j].dy, k), xh = (elem<DT>(cur[j].x, k) - mean) * rstd, g = dy * w[j][k];
        c1 += g;
        c2 = __builtin_fmaf(g, xh, c2);
        dw[j][k] = __builtin_fmaf(dy, xh, dw[j][k]);
        db[j][k] += dy;
      }
    }
    c1 = wave_sum(c1);
    c2 = wave_sum(c2);
    if constexpr (WAVES > 1) {
      if ((t & 63) == 0) red[flip][0][wave] = c1, red[flip][1][wave] = c2;
      lds_barrier();
      c1 = c2 = 0.f;
#pragma unroll
      for (int u = 0; u < WAVES; u++) c1 += red[flip][0][u], c2 += red[flip][1][u];
    }
    c1 *= k1;
    c2 *= k1;
    E* dx = reinterpret_cast<E*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const int64_t c = (int64_t)(j * T + t) * 8;
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float xh = (elem<DT>(cur[j].x, k) - mean) * rstd, g = elem<DT>(cur[j].dy, k) * w[j][k];
        o[k] = rstd * (g - c1 - xh * c2);
      }
      if (c < p.K) store8<DT>(dx, c, p.K, o);
      if constexpr (AHEAD) cur[j] = next[j];
    }
    if constexpr (AHEAD)
      mean = mu, rstd = rs;
    else
      load(cur, row + step, mean, rstd);
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.x * 2 * p.K;
  if constexpr (RPB > 1) {
    // the block's rows were taken by RPB waves: their sums, in order
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
      for (int k = 0; k < 8; k++) {
        wide[((sub * NV + j) * 16 + k) * T + t] = dw[j][k];
        wide[((sub * NV + j) * 16 + 8 + k) * T + t] = db[j][k];
      }
    __syncthreads();
    if (sub) return;
    for (int u = 1; u < RPB; u++)
#pragma unroll
      for (int j = 0; j < NV; j++)
#pragma unroll
        for (int k = 0; k < 8; k++) {
          dw[j][k] += wide[((u * NV + j) * 16 + k) * T + t];
          db[j][k] += wide[((u * NV + j) * 16 + 8 + k) * T + t];
        }
  }
#pragma unroll
  for (int j = 0; j < NV; j++) {
    const int64_t c = (int64_t)(j * T + t) * 8;
    if (c >= p.K) continue;
    store8<MxF32>(out, c, p.K, dw[j]);
    store8<MxF32>(out + p.K, c, p.K, db[j]);
  }
}

// Rows of any length: dx alone, dy and x read twice.
template <class DT>
__global__ __launch_bounds__(1024) void k_norm_grad_long(NormGradParams p) {
  typedef typename DT::T E;
  __shared__ float red[2][2][16];
  const int t = threadIdx.x, wave = t >> 6;
  const float k1 = 1.f / (float)p.K;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, flip ^= 1) {
    const E *dy = reinterpret_cast<const E*>(p.dy) + row * p.lddy, *x = reinterpret_cast<const E*>(p.x) + row * p.ldx;
    E* dx = reinterpret_cast<E*>(p.dx) + row * p.lddx;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float c1 = 0.f, c2 = 0.f;
    for (int64_t c = (int64_t)t * 8; c < p.K; c += 8192) {
      const Vec8<DT> a = load8<DT>(dy, c, p.K);
      Vec8<DT> b = load8<DT>(x, c, p.K);
      repeat8<DT>(b, p.K - c);
      float w[8];
      param8<DT>(w, p.weight, p.param_f32, c, p.K, 1.f);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float g = elem<DT>(a, k) * w[k];
        c1 += g;
        c2 = __builtin_fmaf(g, (elem<DT>(b, k) - mean) * rstd, c2);
      }
    }
    c1 = wave_sum(c1);
    c2 = wave_sum(c2);
    if ((t & 63) == 0) red[flip][0][wave] = c1, red[flip][1][wave] = c2;
    __syncthreads();
    c1 = c2 = 0.f;
#pragma unroll
    for (int u = 0; u < 16; u++) c1 += red[flip][0][u], c2 += red[flip][1][u];
    c1 *= k1;
    c2 *= k1;
    for (int64_t c = (int64_t)t * 8; c < p.K; c += 8192) {
      const Vec8<DT> a = load8<DT>(dy, c, p.K), b = load8<DT>(x, c, p.K);
      float w[8], o[8];
      param8<DT>(w, p.weight, p.param_f32, c, p.K, 1.f);
#pragma unroll
      for (int k = 0; k < 8; k++) o[k] = rstd * (elem<DT>(a, k) * w[k] - c1 - (elem<DT>(b, k) - mean) * rstd * c2);
      store8<DT>(dx, c, p.K, o);
    }
  }
}

// Partial dweight and dbias of strip `blockIdx.y` of rows, for rows of any length: 512 columns a block, a wave a row.
template <class DT>
__global__ __launch_bounds__(256) void k_norm_grad_cols(NormGradParams p, float* part, int64_t strip_rows) {
  typedef typename DT::T E;
  __shared__ float sum[4][2][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 512 + 8 * lane;
  const int64_t r0 = blockIdx.y * strip_rows, r1 = min(r0 + strip_rows, p.M);
  float dw[8] = {}, db[8] = {};
  for (int64_t r = r0 + wave; r < r1; r += 4) {
    const Vec8<DT> a = load8<DT>(reinterpret_cast<const E*>(p.dy) + r * p.lddy, c, p.K);
    const Vec8<DT> b = load8<DT>(reinterpret_cast<const E*>(p.x) + r * p.ldx, c, p.K);
    const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const float dy = elem<DT>(a, k);
      dw[k] = __builtin_fmaf(dy, (elem<DT>(b, k) - mean) * rstd, dw[k]);
      db[k] += dy;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; k++) sum[wave][0][8 * lane + k] = dw[k], sum[wave][1][8 * lane + k] = db[k];
  __syncthreads();
  for (int i = threadIdx.x; i < 1024; i += 256) {
    const int64_t col = (int64_t)blockIdx.x * 512 + (i & 511);
    const int which = i >> 9, at = i & 511;
    if (col >= p.K) continue;
    part[((int64_t)blockIdx.y * 2 + which) * p.K + col] =
        (sum[0][which][at] + sum[1][which][at]) + (sum[2][which][at] + sum[3][which][at]);
  }
}

// The blocks' sums, added by 16 waves: four at a time in float32, these in binary64 (each alone takes 0.3 us more of 4.5 with 512 parts, for its
// conversions). 64 columns a block.
template <class DT>
__global__ __launch_bounds__(1024) void k_norm_join(const float* part, int parts, int64_t K, void* dweight, void* dbias) {
  typedef typename DT::T E;
  __shared__ double sum[16][2][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane, c = col < K ? col : K - 1;
  double a = 0, b = 0;
  for (int k = wave; k < parts; k += 64) {
    float u[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float* at = part + (int64_t)min(k + 16 * i, parts - 1) * 2 * K + c;
      u[i] = at[0], v[i] = at[K];
    }
#pragma unroll
    for (int i = 1; i < 4; i++)
      if (k + 16 * i >= parts) u[i] = v[i] = 0.f;
    a += (double)((u[0] + u[1]) + (u[2] + u[3]));
    b += (double)((v[0] + v[1]) + (v[2] + v[3]));
  }
  sum[wave][0][lane] = a;
  sum[wave][1][lane] = b;
  __syncthreads();
  if (wave > 1 || col >= K) return;
  double s = 0;
#pragma unroll
  for (int w = 0; w < 16; w++) s += sum[w][wave][lane];
  reinterpret_cast<E*>(wave ? dbias : dweight)[col] = DT::store((float)s);
}

}  // namespace dev

using namespace dev;

constexpr int64_t kMostBlocks = 1 << 20;  // of kernels that walk over what is left
static unsigned blocks_of(int64_t n) { return (unsigned)(n < kMostBlocks ? n : kMostBlocks); }

template <class DT, int T, int NV, int OUT>
static void launch_rows(const NormParams& p, hipStream_t stream) {
  constexpr int RPB = T < 256 ? 256 / T : 1;
  const int64_t blocks = (p.M + RPB - 1) / RPB, most = 1024 * 256 / (T < 256 ? 256 : T);  // as many as the chip holds at once
  k_norm<DT, T, NV, OUT><<<(unsigned)(blocks < most ? blocks : most), T < 256 ? 256 : T, 0, stream>>>(p);
}

template <class DT, int OUT>
static hipError_t norm_t(const NormParams& p, hipStream_t stream) {
  const int64_t Kp = OUT == NORM_Y ? p.K : (OUT == NORM_I8 ? (int64_t)p.i8.kq * 64 : (int64_t)p.mx.kq * 128);
  // Two vectors a thread; four of 256 threads past 4096 columns where there are many rows, unless their codes wait for a second
  // maximum or float32 rows leave as float32. Four of 256 and two of 512, us: bf16 1024 x 5003 14.7 and 10.5, 4096 x 5003 32.6 and 30.1,
  // 6000 x 6144 39.0 and 40.7, 8192 x 8192 51.7 and 54.0, 16384 x 6144 90 and 99; to MXFP4 2048 x 5003 18.4 and 17.2, 3000 x 6144 23.1 and 23.9, 8192 x
  // 8192 51.9 and 57.7; to 8 bits 8192 x 5003 71 and 69, 8192 x 8192 68.0 and 68.9; float32 4096 x 8192 52.2 and 50.2, 16384 x 8192 204 and 193, to
  // MXFP4 4096 x 5003 34.9 and 31.8, 8192 x 8192 67.2 and 67.4, 16384 x 6144 111 and 117. (One of 1024: 8192 x 8192 bf16 68, to 8 bits 94.) Three of
  // 512 past 8192 columns: 8192 x 12288 bf16 87 us, two of 1024 107, to 8 bits 120 and 132
  constexpr bool four = OUT == NORM_MX || (OUT == NORM_Y && DT::size == 2);
  constexpr int64_t many = DT::size == 4 ? 8192 : (OUT == NORM_MX ? 3000 : 5000);
  if (p.K < 8)
    launch_rows<DT, 1024, 0, OUT>(p, stream);
  else if (Kp <= 512)
    launch_rows<DT, 64, 1, OUT>(p, stream);
  else if (Kp <= 1024)
    launch_rows<DT, 64, 2, OUT>(p, stream);
  else if (Kp <= 2048)
    launch_rows<DT, 128, 2, OUT>(p, stream);
  else if (Kp <= 4096)
    launch_rows<DT, 256, 2, OUT>(p, stream);
  else if (Kp <= 8192) {
    if constexpr (four)
      if (p.M > many) {
        launch_rows<DT, 256, 4, OUT>(p, stream);
        return hipGetLastError();
      }
    launch_rows<DT, 512, 2, OUT>(p, stream);
  } else if (Kp <= 12288)
    launch_rows<DT, 512, 3, OUT>(p, stream);
  else if (Kp <= 16384)
    launch_rows<DT, 1024, 2, OUT>(p, stream);
  else
    launch_rows<DT, 1024, 0, OUT>(p, stream);
  return hipGetLastError();
}

template <class DT>
static hipError_t norm_dt(const NormParams& p, hipStream_t stream) {
  if (p.i8.codes) return norm_t<DT, NORM_I8>(p, stream);
  if (p.mx.codes) return norm_t<DT, NORM_MX>(p, stream);
  return norm_t<DT, NORM_Y>(p, stream);
}

hipError_t launch_norm(const NormParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case SVDQ_F32: return norm_dt<MxF32>(p, stream);
    case SVDQ_BF16: return norm_dt<MxBF16>(p, stream);
    default: return norm_dt<MxF16>(p, stream);
  }
}

// Rows whose columns a block's threads do not keep: longer than their registers, or shorter than a vector.
static bool apart(int64_t K) { return K > 16384 || K < 8; }

// Rows that a wave adds up in float32, at most (more only where a grid would pass 65535 strips: 2^28 rows). A longer chain's error grows with
// the rows.
constexpr int64_t kChain = 1024;

// Blocks of a launch (or strips of rows) that leave a part of dweight and dbias each.
static int64_t grad_blocks(int64_t M, int64_t K) {
  if (apart(K)) {
    int64_t strips = (M + 15) / 16;
    if (strips > 64) strips = 64;
    const int64_t least = (M + 4 * kChain - 1) / (4 * kChain);
    if (strips < least) strips = least < 65535 ? least : 65535;
    const int64_t rows = (M + strips - 1) / strips;
    return (M + rows - 1) / rows;
  }
  // 8192 x 8192 bf16 with 128, 256 and 512 parts 98, 80 and 86 us, 8192 x 2048 53, 33 and 28, 515 x 2731 11.3, 12.2 and 16.9
  const int64_t rows = K <= 512 ? 4 : 1, most = K <= 2048 ? 512 : 256;  // of a block at once
  int64_t parts = (M + 4 * rows - 1) / (4 * rows);
  if (parts > most) parts = most;
  if (parts < 64) parts = (M + rows - 1) / rows < 64 ? (M + rows - 1) / rows : 64;
  return parts;
}

// Launches, of as many rows each. (As many more blocks in one launch instead: its last round does not fill the chip, 600000 x 4096 bf16 3.0 to
// 3.7 ms and in three launches 2.7. Parts that a block leaves on its way: the kernel's registers, 122 of them spilled in rows of 16384.)
static int64_t grad_runs(int64_t M, int64_t K) {
  if (apart(K)) return 1;
  const int64_t most = grad_blocks(M, K) * (K <= 512 ? 4 : 1) * kChain;
  return (M + most - 1) / most;
}
static int64_t grad_parts(int64_t M, int64_t K) { return grad_blocks(M, K) * grad_runs(M, K); }

size_t norm_grad_bytes(int64_t M, int64_t K, bool params) { return params ? (size_t)(grad_parts(M, K) * 2 * K * 4 + 255) / 256 * 256 : 0; }

bool norm_grad_fits(int64_t K) { return mx_fits_grid((K + 63) / 64, 1024); }

template <class DT, int T, int NV, bool AHEAD = true>
static void launch_grad(const NormGradParams& p, float* part, hipStream_t stream) {
  const int64_t blocks = grad_blocks(p.M, p.K), runs = grad_runs(p.M, p.K), rows = (p.M + runs - 1) / runs;
  for (int64_t k = 0; k < runs; k++) {
    const int64_t r = k * rows;
    NormGradParams q = p;
    q.dy = reinterpret_cast<const typename DT::T*>(p.dy) + r * p.lddy;
    q.x = reinterpret_cast<const typename DT::T*>(p.x) + r * p.ldx;
    q.dx = reinterpret_cast<typename DT::T*>(p.dx) + r * p.lddx;
    q.mean = p.mean + r;
    q.rstd = p.rstd + r;
    q.M = rows < p.M - r ? rows : p.M - r;
    k_norm_grad<DT, T, NV, AHEAD><<<(unsigned)blocks, T < 256 ? 256 : T, 0, stream>>>(q, part ? part + k * blocks * 2 * p.K : nullptr);
  }
}

template <class DT>
static hipError_t grad_t(const NormGradParams& p, hipStream_t stream) {
  float* part = p.weight ? reinterpret_cast<float*>(p.workspace) : nullptr;
  const int64_t parts = grad_parts(p.M, p.K);
  if (apart(p.K)) {
    k_norm_grad_long<DT><<<blocks_of(p.M), 1024, 0, stream>>>(p);
    if (part)
      k_norm_grad_cols<DT><<<dim3((unsigned)((p.K + 511) / 512), (unsigned)parts), 256, 0, stream>>>(p, part, (p.M + parts - 1) / parts);
  } else if (p.K <= 512) {
    launch_grad<DT, 64, 1>(p, part, stream);
  } else if (p.K <= 2048) {
    launch_grad<DT, 256, 1>(p, part, stream);
  } else if (p.K <= 4096) {
    launch_grad<DT, 512, 1>(p, part, stream);
  } else if (p.K <= 8192) {
    launch_grad<DT, 512, 2>(p, part, stream);
  } else if (p.K <= 12288) {
    launch_grad<DT, 512, 3>(p, part, stream);
  } else {
    launch_grad<DT, 512, 4, false>(p, part, stream);
  }
  if (part) {
    const unsigned blocks = (unsigned)((p.K + 63) / 64);
    if (p.param_f32)
      k_norm_join<MxF32><<<blocks, 1024, 0, stream>>>(part, (int)parts, p.K, p.dweight, p.dbias);
    else
      k_norm_join<DT><<<blocks, 1024, 0, stream>>>(part, (int)parts, p.K, p.dweight, p.dbias);
  }
  return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case SVDQ_F32: return grad_t<MxF32>(p, stream);
    case SVDQ_BF16: return grad_t<MxBF16>(p, stream);
    default: return grad_t<MxF16>(p, stream);
  }
}

}  // namespace svdq
