// Device helpers of the MXFP4-tensor kernels: storage types with conversions that keep NaN,
// eight codes at a time from packed values, and the gated activations with their derivatives.
#pragma once

#include <type_traits>

#include "device_common.h"

#include "../../include/svdq.h"

namespace svdq {
namespace dev {

// Storage types: `pair` is two 16-bit values in one word (the lower index in the low half); wide: a product of two values may
// pass the float32 range.
struct MxF32 {
  typedef float T;
  static constexpr int size = 4;
  static constexpr bool wide = true;
  __device__ static inline float load(T v) { return v; }
  __device__ static inline T store(float v) { return v; }
};
struct MxBF16 {
  typedef uint16_t T;
  static constexpr int size = 2;
  static constexpr bool wide = true;
  __device__ static inline float load(T v) { return __uint_as_float((u32)v << 16); }
  __device__ static inline T store(float v) { return (T)pack_bf16x2(v, v); }
  __device__ static inline u32 pack(float a, float b) { return pack_bf16x2(a, b); }
  // v_cvt_scalef32_pk_fp4_bf16 over four pairs, see fp4_pack8_bf16
  __device__ static inline u32 codes8(const u32* pairs, float scale) { return fp4_pack8_bf16(pairs, scale); }
};
struct MxF16 {
  typedef uint16_t T;
  static constexpr int size = 2;
  static constexpr bool wide = false;
  __device__ static inline float load(T v) { return (float)__builtin_bit_cast(_Float16, v); }
  __device__ static inline T store(float v) { return __builtin_bit_cast(T, (_Float16)v); }
  __device__ static inline u32 pack(float a, float b) { return (u32)store(a) | ((u32)store(b) << 16); }
  __device__ static inline u32 codes8(const u32* pairs, float scale) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    u32 r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, pairs[0]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, pairs[1]), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, pairs[2]), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, pairs[3]), scale, 3);
    return r;
  }
};

// Scale byte e + 127 of a block from the bits of its largest magnitude as float32, with e the smallest with amax <=
// 6 * 2^e = 1.5 * 2^(e + 2): the exponent field, one more where the fraction is past 1/2, less 2; 0 below 2^-126; 255 (NaN)
// from infinity on.
__device__ inline u32 mx_scale_byte(u32 amax_bits) {
  const u32 e = max((amax_bits + 0x3FFFFFu) >> 23, 2u) - 2u;
  return amax_bits >= 0x7F800000u ? 255u : e;
}
// 2^e of a scale byte below 255.
__device__ inline float mx_scale_value(u32 byte) { return __uint_as_float(max(byte << 23, 0x00400000u)); }

// ---- eight elements at a time ------------------------------------------------------------
// Eight consecutive elements of a row, in registers.
template <class DT>
struct Vec8 {
  u32 w[DT::size * 2];  // 16-bit types: four pairs; float32: eight values' bits
};

template <class DT>
__device__ inline Vec8<DT> zero8() {
  Vec8<DT> v;
#pragma unroll
  for (int q = 0; q < DT::size * 2; q++) v.w[q] = 0;
  return v;
}

// Elements [c, c + 8) of a row of C elements at src, zeros past its end. A whole vector is loaded
// at any alignment of its elements (global loads need none on this target).
template <class DT>
__device__ inline Vec8<DT> load8(const typename DT::T* src, int64_t c, int64_t C) {
  Vec8<DT> v = zero8<DT>();
  if (c + 8 <= C) {
    __builtin_memcpy(&v, src + c, sizeof v);
  } else {
#pragma unroll
    for (int q = 0; q < 8; q++) {
      if (c + q >= C) continue;
      if constexpr (DT::size == 4)
        v.w[q] = __float_as_uint(src[c + q]);
      else
        v.w[q >> 1] |= (u32)src[c + q] << (16 * (q & 1));
    }
  }
  return v;
}

template <class DT>
__device__ inline float elem(const Vec8<DT>& v, int q) {
  if constexpr (DT::size == 4)
    return __uint_as_float(v.w[q]);
  else
    return DT::load((uint16_t)(v.w[q >> 1] >> (16 * (q & 1))));
}

typedef uint16_t v2us __attribute__((ext_vector_type(2)));

// Largest magnitude of packed 16-bit values: magnitudes order as their bits do.
__device__ inline u32 max_pairs(u32 a, u32 b) {
  return __builtin_bit_cast(u32, __builtin_elementwise_max(__builtin_bit_cast(v2us, a), __builtin_bit_cast(v2us, b)));
}

// Bits of the largest magnitude of n words of a block's share, as float32.
template <class DT, int N>
__device__ inline u32 amax_bits(const u32 (&w)[N]) {
  if constexpr (DT::size == 4) {
    u32 m = 0;
#pragma unroll
    for (int q = 0; q < N; q++) m = max(m, w[q] & 0x7FFFFFFFu);
    return m;
  } else {
    u32 m = 0;
#pragma unroll
    for (int q = 0; q < N; q++) m = max_pairs(m, w[q] & 0x7FFF7FFFu);
    return __float_as_uint(DT::load((uint16_t)max(m & 0xFFFFu, m >> 16)));
  }
}

// The word of eight codes (zeros for a NaN block).
template <class DT>
__device__ inline u32 codes8(const u32* w, u32 byte) {
  const float s = mx_scale_value(byte);
  u32 c;
  if constexpr (DT::size == 4) {
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; q++) v[q] = __uint_as_float(w[q]);
    c = fp4_pack8(v, s);
  } else {
    c = DT::codes8(w, s);
  }
  return byte == 255u ? 0u : c;
}

// ---- gated activations ------------------------------------------------------------------
// act(g) and act'(g). For float, with ew, abs_d: |error of act| <= ew |act|, |error of act'| <= abs_d, good while
// tail >= -60 (below that a factor nears the bottom of the float32 range):
//   silu       g s,  s = 1 / (1 + e^-w), w = g
//   gelu_tanh  g s with w = 2 sqrt(2 / pi) (g + 0.044715 g^3), which equals
//              g (1 + tanh(w / 2)) / 2 without its cancellation for negative g
//     act' = s (1 + g (1 - s) w'). v_exp_f32 on w log2(e) is off by (2 + |w|) 2^-23 relative,
//     the sigmoid by at most (2 + |w|) 2^-22; 1 - s by that times s absolutely, which g w'
//     multiplies: together act' is within s (1 + |g w'|) (3 + |w|) 2^-21.
//   gelu       g P, P = erfc(-g / sqrt 2) / 2; act' = P + g e^(-g^2 / 2) / sqrt(2 pi). Rounding
//     the argument moves erfc by g^2 2^-24 relative, erfcf and the exponential by a few ulps.
//   relu       max(g, 0), 1 where g > 0
// NaN and infinite g give NaN in at least one of the two.
template <class F>
struct ActValue {
  F a, d;
  float ew, abs_d, tail;
};

__device__ inline float act_exp(float v) { return __expf(v); }
__device__ inline double act_exp(double v) { return exp(v); }
__device__ inline float act_rcp(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ inline double act_rcp(double v) { return 1.0 / v; }
__device__ inline float act_erfc(float v) { return erfcf(v); }
__device__ inline double act_erfc(double v) { return erfc(v); }

template <int ACT, class F>
__device__ inline ActValue<F> act_value(F g) {
  ActValue<F> r;
  if constexpr (ACT == SVDQ_ACT_RELU) {
    const F none = g == g ? F(0) : g;  // +0 for either zero, NaN for a NaN
    r.a = g > F(0) ? g : none;
    r.d = g > F(0) ? F(1) : none;
    r.ew = 0x1p-22f;
    r.abs_d = (float)r.d * 0x1p-22f;
    r.tail = 0.f;
  } else if constexpr (ACT == SVDQ_ACT_GELU) {
    const F p = F(0.5) * act_erfc(F(-0.70710678118654752440) * g);
    const F q = g * (F(0.39894228040143267794) * act_exp(F(-0.5) * g * g));
    r.a = g * p;
    r.d = p + q;
    r.ew = (3.f + (float)(g * g)) * 0x1p-20f;
    r.abs_d = ((float)p + fabsf((float)q)) * r.ew;
    r.tail = 6.f * (float)g;
  } else {
    F w = g, dw = F(1), gc = g;
    if constexpr (ACT == SVDQ_ACT_GELU_TANH) {
      // past 30 the sigmoid is 0 or 1 and w' times 1 - s no longer counts, but g^3 could overflow
      gc = g > F(30) ? F(30) : (g < F(-30) ? F(-30) : g);
      const F c = F(1.59576912160573071176), g2 = gc * gc;
      w = gc * (c + F(1.59576912160573071176 * 0.044715) * g2);
      dw = c + F(1.59576912160573071176 * 0.134145) * g2;
    }
    const F s = act_rcp(F(1) + act_exp(-w)), gw = gc * dw;
    r.a = g * s;
    r.d = s * (F(1) + gw * (F(1) - s));
    r.ew = (3.f + fabsf((float)w)) * 0x1p-21f;
    r.abs_d = (float)s * (1.f + fabsf((float)gw)) * r.ew;
    r.tail = (float)w;
  }
  return r;
}

template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case SVDQ_ACT_SILU: f(std::integral_constant<int, SVDQ_ACT_SILU>()); break;
    case SVDQ_ACT_GELU: f(std::integral_constant<int, SVDQ_ACT_GELU>()); break;
    case SVDQ_ACT_GELU_TANH: f(std::integral_constant<int, SVDQ_ACT_GELU_TANH>()); break;
    default: f(std::integral_constant<int, SVDQ_ACT_RELU>()); break;
  }
}

}  // namespace dev
}  // namespace svdq
