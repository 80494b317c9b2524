// Device helpers of the 8-bit tensor and layer norm kernels: reductions over a wave and a block, and the codes of values.
#pragma once

#include "mx_device.h"

namespace svdq {
namespace dev {

// ---- reductions ---------------------------------------------------------------------------
// Lane exchanges within a row of 16 (DPP): lanes 1, 2, 4 (mirrored halves) and 8 (mirrored row) apart.
template <int CTRL>
__device__ inline u32 dpp(u32 v) {
  return (u32)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kQuad1 = 0xB1, kQuad2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
template <int CTRL>
__device__ inline double dpp(double v) {
  const u64 u = __builtin_bit_cast(u64, v);
  return __builtin_bit_cast(double, (u64)dpp<CTRL>((u32)u) | ((u64)dpp<CTRL>((u32)(u >> 32)) << 32));
}
template <int CTRL>
__device__ inline float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
__device__ inline u32 lane_of(u32 v, int lane) { return (u32)__builtin_amdgcn_readlane((int)v, lane); }
__device__ inline float lane_of(float v, int lane) { return __uint_as_float(lane_of(__float_as_uint(v), lane)); }
__device__ inline double lane_of(double v, int lane) {
  const u64 u = __builtin_bit_cast(u64, v);
  return __builtin_bit_cast(double, (u64)lane_of((u32)u, lane) | ((u64)lane_of((u32)(u >> 32), lane) << 32));
}

// Two sums that travel together.
struct __align__(16) Sums2 {
  double a, b;
};
template <int CTRL>
__device__ inline Sums2 dpp(const Sums2& v) {
  return {dpp<CTRL>(v.a), dpp<CTRL>(v.b)};
}
__device__ inline Sums2 lane_of(const Sums2& v, int lane) { return {lane_of(v.a, lane), lane_of(v.b, lane)}; }
__device__ inline Sums2 add2(const Sums2& u, const Sums2& v) { return {u.a + v.a, u.b + v.b}; }
__device__ inline u32 umax2(u32 a, u32 b) { return max(a, b); }

// Over the 16 lanes of a row (all lanes of the wave active), the same value in each of them; `add` joins two values.
template <class V, class F>
__device__ inline V row_join(V v, F add) {
  v = add(v, dpp<kQuad1>(v));
  v = add(v, dpp<kQuad2>(v));
  v = add(v, dpp<kHalfMirror>(v));
  return add(v, dpp<kMirror>(v));
}
// Over all 64 lanes of a wave, the same value in every lane.
template <class V, class F>
__device__ inline V wave_join(V v, F add) {
  v = row_join(v, add);
  return add(add(lane_of(v, 0), lane_of(v, 16)), add(lane_of(v, 32), lane_of(v, 48)));
}
template <class V>
__device__ inline V wave_sum(V v) {
  return wave_join(v, [](V a, V b) { return a + b; });
}
__device__ inline u32 wave_umax(u32 v) {
  return wave_join(v, umax2);
}

// Over the waves (2, 4, 8 or 16) that share a row, from what `row_join` left for each 16 of their threads, in LDS: four values a wave. A lane
// takes every sixteenth, and every group of lanes that the steps below join has them all.
template <int WAVES, class V, class F>
__device__ inline V waves_join(const V* part, F add) {
  static_assert(WAVES == 2 || WAVES == 4 || WAVES == 8 || WAVES == 16, "whole groups of lanes");
  constexpr int LANES = WAVES < 4 ? 4 * WAVES : 16;
  V v = part[threadIdx.x & (LANES - 1)];
#pragma unroll
  for (int k = 1; k < WAVES / 4; k++) v = add(v, part[(threadIdx.x & 15) + 16 * k]);
  v = add(v, dpp<kQuad1>(v));
  v = add(v, dpp<kQuad2>(v));
  v = add(v, dpp<kHalfMirror>(v));
  if constexpr (LANES == 16) v = add(v, dpp<kMirror>(v));
  return v;
}

// ---- elements of a row --------------------------------------------------------------------
// Elements [c, c + 8) of a row of K >= 8, whole vectors without a branch: where they pass the row's end, its last eight, which
// `fit8` moves into place, with `past` (bits of an element) behind them. Only waves at a row's end take that branch.
template <class DT>
__device__ inline Vec8<DT> load8_last(const typename DT::T* row, int64_t c, int64_t K) {
  Vec8<DT> v;
  __builtin_memcpy(&v, row + (c < K - 8 ? c : K - 8), sizeof v);
  return v;
}
template <class DT>
__device__ inline void fit8(Vec8<DT>& v, int64_t c, int64_t K, u32 past = 0) {
  if (!__builtin_amdgcn_ballot_w64(c + 8 > K)) return;
  const int s = (int)(c + 8 <= K ? 0 : (c < K ? c + 8 - K : 8));  // elements to move down by
  constexpr int W = DT::size * 2, E = W / 4;                      // words of a vector, of two elements
  const u32 fill = DT::size == 4 ? past : past * 0x10001u;
#pragma unroll
  for (int k = 0; k < W; k++) v.w[k] = s & 8 ? fill : v.w[k];
#pragma unroll
  for (int k = 0; k < W; k++) v.w[k] = s & 4 ? (k + 2 * E < W ? v.w[(k + 2 * E) % W] : fill) : v.w[k];
#pragma unroll
  for (int k = 0; k < W; k++) v.w[k] = s & 2 ? (k + E < W ? v.w[(k + E) % W] : fill) : v.w[k];
#pragma unroll
  for (int k = 0; k < W; k++) {
    const u32 up = k + 1 < W ? v.w[(k + 1) % W] : fill;
    v.w[k] = s & 1 ? (DT::size == 4 ? up : (v.w[k] >> 16) | (up << 16)) : v.w[k];
  }
}

// The same where the places past the row's end keep elements of the row, for what a product with 0 must take back out: they are infinite or
// NaN only if the row's own are.
template <class DT>
__device__ inline void turn8(Vec8<DT>& v, int64_t c, int64_t K) {
  if (!__builtin_amdgcn_ballot_w64(c + 8 > K)) return;
  const int s = c + 8 <= K || c >= K ? 0 : (int)(c + 8 - K);  // elements to move down by, as masks for each power of two
  const u32 m4 = 0u - (u32)(s >> 2 & 1), m2 = 0u - (u32)(s >> 1 & 1), m1 = 0u - (u32)(s & 1);
  auto pick = [](u32 m, u32 a, u32 b) { return (a & m) | (b & ~m); };
  constexpr int W = DT::size * 2, E = W / 4;
#pragma unroll
  for (int k = 0; k < W - 2 * E; k++) v.w[k] = pick(m4, v.w[k + 2 * E], v.w[k]);
#pragma unroll
  for (int k = 0; k < W - E; k++) v.w[k] = pick(m2, v.w[k + E], v.w[k]);
#pragma unroll
  for (int k = 0; k < W; k++) {
    const u32 up = v.w[k + 1 < W ? k + 1 : k];
    v.w[k] = pick(m1, DT::size == 4 ? up : (v.w[k] >> 16) | (k + 1 < W ? up << 16 : up & 0xFFFF0000u), v.w[k]);
  }
}
// And of a vector of which the first n elements, one at least, are the row's.
template <class DT>
__device__ inline void repeat8(Vec8<DT>& v, int64_t n) {
  if (n >= 8) return;
  const u32 first = DT::size == 4 ? v.w[0] : v.w[0] & 0xFFFFu;
#pragma unroll
  for (int q = 1; q < 8; q++) {
    if (q < n) continue;
    if constexpr (DT::size == 4)
      v.w[q] = first;
    else
      v.w[q >> 1] = q & 1 ? (v.w[q >> 1] & 0xFFFFu) | (first << 16) : (v.w[q >> 1] & 0xFFFF0000u) | first;
  }
}

// Elements [c, c + 8) of a row of K.
template <class DT>
__device__ inline void store8(typename DT::T* row, int64_t c, int64_t K, const float (&v)[8]) {
  if (c + 8 <= K) {
    u32 o[DT::size * 2];
#pragma unroll
    for (int q = 0; q < DT::size * 2; q++) {
      if constexpr (DT::size == 4)
        o[q] = __float_as_uint(v[q]);
      else
        o[q] = DT::pack(v[2 * q], v[2 * q + 1]);
    }
    __builtin_memcpy(row + c, o, sizeof o);
  } else {
#pragma unroll
    for (int k = 0; k < 8; k++)
      if (c + k < K) row[c + k] = DT::store(v[k]);
  }
}

// ---- 8-bit codes --------------------------------------------------------------------------
// A row's scale from the bits of its largest magnitude: float32(max / 127), 2^-126 at least (so that every step below is
// exact), 0 for a row of zeros, NaN if the row holds an infinity or a NaN.
struct Scale8 {
  float s;  // as stored
  float r;  // float32(1 / s); 0 where every code is 0
};
__device__ inline Scale8 scale8(u32 amax_bits) {
  if (amax_bits >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), 0.f};
  if (amax_bits == 0) return {0.f, 0.f};
  const float s = fmaxf(__uint_as_float(amax_bits) / 127.0f, 0x1p-126f);
  return {s, 1.0f / s};
}

// The nearest integer to x / s, ties to even, in the low byte of u.
// x r differs from x / s by less than 2^-16.9, so adding 1.5 * 2^23 to it (one rounding, to an integer k) gives that integer or, next
// to a border, its neighbour. The remainder x - k s, which one fma gives exactly, says which: k is right if its double is smaller than s in
// size, or equal and k even. (Exactly: the remainder is a multiple of the smaller unit of x and s, and at most s / 2 (1 + 2^-15). It is
// doubled, and not s halved: half of a scale below 2^-125 may be no float32.)
// Borders are no rare case in 16-bit types, whose x 127 / max are often half a whole number but for the rounding of s: the
// test of a vector costs one operation an element, mending it seven more.
constexpr float kMagic8 = 12582912.f;
struct Code8 {
  float u, rem;
};
__device__ inline Code8 code8(float x, float s, float r, float& far) {
  const float u = __builtin_fmaf(x, r, kMagic8), rem = __builtin_fmaf(kMagic8 - u, s, x);
  far = fmaxf(far, fabsf(rem));
  return {u, rem};
}
// Whether a vector holds an element at a border or past it, from the largest of its remainders.
__device__ inline bool border8(float far, float s) { return far + far >= s; }
__device__ inline void mend8(Code8& c, float s) {
  // 2 |rem| > s, or equal where k is odd: by their bits
  const bool off = (__float_as_uint(c.rem + c.rem) & 0x7FFFFFFFu) + (__float_as_uint(c.u) & 1u) > __float_as_uint(s);
  c.u += off ? copysignf(1.f, c.rem) : 0.f;
}
__device__ inline u32 bytes4(float a, float b, float c, float d) {
  const u32 lo = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x0C0C0400u);
  const u32 hi = __builtin_amdgcn_perm(__float_as_uint(d), __float_as_uint(c), 0x04000C0Cu);
  return lo | hi;
}

// Eight codes of v[0..7], in order.
__device__ inline v2u codes8x8(const float (&v)[8], const Scale8& q) {
  Code8 c[8];
  float far = 0.f;
#pragma unroll
  for (int k = 0; k < 8; k++) c[k] = code8(v[k], q.s, q.r, far);
  if (__builtin_amdgcn_ballot_w64(border8(far, q.s))) {
#pragma unroll
    for (int k = 0; k < 8; k++) mend8(c[k], q.s);
  }
  const v2u w = {bytes4(c[0].u, c[1].u, c[2].u, c[3].u), bytes4(c[4].u, c[5].u, c[6].u, c[7].u)};
  return q.r == 0.f ? v2u{0, 0} : w;
}

// Whether a scale may enter a float32 product with another such scale and an int32 without leaving the normal range.
__device__ inline bool tame(float s) { return s == 0.f || (s >= 0x1p-60f && s <= 0x1p40f); }

// y from a sum and its scales, the same in every kernel: in float32 where they are tame, else in binary64 (an infinite product of scales would make a NaN
// of a zero sum, a vanished one a zero of a large sum). Which of them depends on the output's own scales alone.
__device__ inline float scaled(int sum, float sa, float sb, float bias) { return __builtin_fmaf((float)sum, sa * sb, bias); }
__device__ inline float scaled_far(int sum, float sa, float sb, float bias) {
  if (tame(sa) && tame(sb)) return scaled(sum, sa, sb, bias);
  return (float)__builtin_fma((double)sum * (double)sa, (double)sb, (double)bias);
}
// Of a sum that may pass 32 bits.
__device__ inline float scaled_long(int64_t sum, float sa, float sb, float bias) {
  if (sum == (int)sum) return scaled_far((int)sum, sa, sb, bias);
  return (float)__builtin_fma((double)sum * (double)sa, (double)sb, (double)bias);
}

// Where code k of row r lies.
__device__ inline int64_t i8_at(int64_t r, int64_t k, int kq) { return (((r >> 4) * kq + (k >> 6)) << 10) + ((r & 15) << 6) + (k & 63); }

}  // namespace dev
}  // namespace svdq
