// Products of MXFP4 tensors on gfx950: Y = D(A B^T + bias), and the gated projections
// h = D(act(A Wg^T) * (A Wu^T)) of a feed-forward block.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 K-consecutive E2M1 codes per lane (16 bytes) with the
// lane's own E8M0 byte: exactly one block of an MXFP4 tensor. Products of codes and their scales are
// exact; sums are float32.
//
// Simplest form: a wave owns a 32 x 32 output tile and reads its operands straight from memory.
#include <type_traits>

#include "mx.h"
#include "mx_device.h"

namespace svdq {
namespace dev {

template <class F>
__device__ inline void with_act(int act, F f) {
  switch (act) {
    case SVDQ_ACT_SILU: f(std::integral_constant<int, SVDQ_ACT_SILU>()); break;
    case SVDQ_ACT_GELU: f(std::integral_constant<int, SVDQ_ACT_GELU>()); break;
    case SVDQ_ACT_GELU_TANH: f(std::integral_constant<int, SVDQ_ACT_GELU_TANH>()); break;
    default: f(std::integral_constant<int, SVDQ_ACT_RELU>()); break;
  }
}

template <class DT, bool GATED>
__global__ __launch_bounds__(256) void k_mx_product(MxGemmParams p, int tiles_n) {
  typedef typename DT::T T;
  const int t = threadIdx.x, lane = t & 63, l32 = lane & 31, g = lane >> 5;
  const int64_t id = (int64_t)blockIdx.x * 4 + (t >> 6);
  const int64_t tm = id / tiles_n;
  const int64_t m0 = tm * 32, n0 = (id - tm * tiles_n) * 32;
  if (m0 >= p.M) return;
  const int64_t row = m0 + l32 < p.M ? m0 + l32 : p.M - 1;
  const int64_t col = n0 + l32 < p.N ? n0 + l32 : p.N - 1;
  const uint8_t* ac = p.a_codes + (((row >> 4) * p.kq) << 10) + ((row & 15) << 6) + g * 16;
  const uint8_t* as = p.a_scales + mx_scale_tiled_index(row, 0, p.kq) + g;
  const uint8_t *bc[2], *bs[2];
  for (int h = 0; h < (GATED ? 2 : 1); h++) {
    const int64_t br = col + (int64_t)h * p.N;
    bc[h] = p.b_codes + mx_code_tile_offset(br, p.kq) + g * 16;
    bs[h] = p.b_scales + mx_scale_tiled_index(br, 0, p.kq) + g;
  }
  v16f acc[2];
  for (int v = 0; v < 16; v++) acc[0][v] = acc[1][v] = 0.f;
  for (int s = 0; s < p.kq; s++) {
#pragma unroll
    for (int ks = 0; ks < 2; ks++) {
      const v4i a = *reinterpret_cast<const v4i*>(ac + (int64_t)s * 1024 + 32 * ks);
      const int sa = as[(int64_t)s * 256 + 2 * ks];
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); h++) {
        const v4i b = *reinterpret_cast<const v4i*>(bc[h] + (int64_t)s * 1024 + 32 * ks);
        const int sb = bs[h][(int64_t)s * 256 + 2 * ks];
        acc[h] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                                 v8i{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, acc[h], 4, 4, 0,
                                                                 sa, 0, sb);
      }
    }
  }
  if (n0 + l32 >= p.N) return;
  T* y = reinterpret_cast<T*>(p.y) + n0 + l32;
  float bias = 0.f;
  if (!GATED && p.bias) bias = DT::load(reinterpret_cast<const T*>(p.bias)[n0 + l32]);
#pragma unroll
  for (int v = 0; v < 16; v++) {
    const int64_t r = m0 + 8 * (v / 4) + 4 * g + (v % 4);
    if (r >= p.M) continue;
    if constexpr (GATED) {
      float a = 0.f;
      with_act(p.act, [&](auto c) { a = act_value<decltype(c)::value, float>(acc[0][v]).a; });
      y[r * p.ldy] = DT::store(a * acc[1][v]);
      if (p.gu) {
        T* gu = reinterpret_cast<T*>(p.gu) + r * p.ldgu + n0 + l32;
        gu[0] = DT::store(acc[0][v]);
        gu[p.N] = DT::store(acc[1][v]);
      }
    } else {
      y[r * p.ldy] = DT::store(acc[0][v] + bias);
    }
  }
}

}  // namespace dev

using namespace dev;

template <class DT>
static hipError_t launch_product_t(const MxGemmParams& p, bool gated, hipStream_t stream) {
  const int64_t tn = (p.N + 31) / 32, tm = (p.M + 31) / 32, blocks = (tn * tm + 3) / 4;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (gated)
    k_mx_product<DT, true><<<dim3((unsigned)blocks), 256, 0, stream>>>(p, (int)tn);
  else
    k_mx_product<DT, false><<<dim3((unsigned)blocks), 256, 0, stream>>>(p, (int)tn);
  return hipGetLastError();
}

hipError_t launch_mx_product(const MxGemmParams& p, bool gated, int dtype, hipStream_t stream) {
  switch (dtype) {
    case SVDQ_F32: return launch_product_t<MxF32>(p, gated, stream);
    case SVDQ_BF16: return launch_product_t<MxBF16>(p, gated, stream);
    default: return launch_product_t<MxF16>(p, gated, stream);
  }
}

}  // namespace svdq
