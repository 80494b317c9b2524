// Pieces shared by the tiled products (k_mx_gemm.hip, k_i8_gemm.hip): the swizzled LDS rows of a stage, record counts
// of buffer resources, and the way a block's tile leaves.
#pragma once

#include "gemm_pipe.h"
#include "mx_device.h"

namespace svdq {
namespace dev {

__device__ inline int lds_swizzle(int row, int chunk) { return row * 64 + ((chunk ^ ((row >> 2) & 3)) << 4); }

__device__ inline int records(int64_t bytes) { return (int)(u32)(bytes < 0xFFFFFFFFll ? bytes : 0xFFFFFFFFll); }

typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));

// Writes a block's tile of VT x values from the lanes of the waves to out[r0 .., c0 ..] (row stride ld, limits rows x
// cols): value(i, j, v) is this lane's accumulator entry of 32 x 32 tile (i, j), of NJ column tiles per
// wave. Rounded, staged through the idle ring and stored 16 bytes a lane (at any alignment). The output is not
// read again here, so it streams past the caches.
template <class DT, class C, int BM, int NJ, class V>
__device__ __forceinline__ void store_tile(uint8_t* smem, typename DT::T* out, int64_t ld, int rows, int cols, int r0,
                                           int c0, int wm, int wn, int lane, V value) {
  typedef typename DT::T T;
  constexpr int W = C::WN * NJ * 32;                                    // tile columns
  constexpr int PH = (BM * W * DT::size + C::SMEM - 1) / C::SMEM;       // phases of BM / PH rows
  static_assert(PH == 1 || PH == 2 || PH == 4, "phases split the wave rows evenly");
  constexpr int PR = BM / PH;
  const int l32 = lane & 31, g = lane >> 5, t = threadIdx.x;
#pragma unroll
  for (int ph = 0; ph < PH; ph++) {
    __syncthreads();
    if (PH == 1 || wm / (C::WM / PH) == ph) {
#pragma unroll
      for (int i = 0; i < C::MT; i++)
#pragma unroll
        for (int j = 0; j < NJ; j++) {
          const int rb = wm * C::TM + 32 * i + 4 * g - ph * PR, cb = wn * NJ * 32 + 32 * j;
          if constexpr (DT::size == 4) {
            float* tile = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int v = 0; v < 16; v++) tile[(rb + 8 * (v / 4) + v % 4) * W + cb + l32] = value(i, j, v);
          } else {
            // rows (r, r + 1) of a column in one word; neighbouring lanes swap words and each keeps one row's
            // pair of columns
            const bool odd = l32 & 1;
            const u32 sel = odd ? 0x03020706u : 0x05040100u;
            uint16_t* tile = reinterpret_cast<uint16_t*>(smem) + (odd ? W : 0) + cb + (l32 & ~1);
#pragma unroll
            for (int v = 0; v < 16; v += 2) {
              const u32 own = DT::pack(value(i, j, v), value(i, j, v + 1));
              const u32 nb = (u32)__builtin_amdgcn_mov_dpp((int)own, 0xB1, 0xF, 0xF, true);
              *reinterpret_cast<u32*>(tile + (rb + 8 * (v / 4) + v % 4) * W) = __builtin_amdgcn_perm(nb, own, sel);
            }
          }
        }
    }
    __syncthreads();
    constexpr int E = 16 / DT::size, CPR = W / E;
    const T* tile = reinterpret_cast<const T*>(smem);
    for (int c = t; c < PR * CPR; c += 64 * C::NWV) {
      const int r = c / CPR, cc = (c - r * CPR) * E;
      const int row = r0 + ph * PR + r, col = c0 + cc;
      if (row >= rows || col >= cols) continue;
      const v4i v = *reinterpret_cast<const v4i*>(tile + r * W + cc);
      T* dst = out + (int64_t)row * ld + col;
      if (col + E <= cols) {
        __builtin_nontemporal_store(v, reinterpret_cast<v4i_any*>(dst));
      } else {
#pragma unroll
        for (int q = 0; q < E; q++)
          if (col + q < cols) dst[q] = tile[r * W + cc + q];
      }
    }
  }
}

}  // namespace dev
}  // namespace svdq
