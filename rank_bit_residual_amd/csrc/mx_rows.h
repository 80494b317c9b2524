// How rows enter an MXFP4 tensor, eight elements per lane (k_mx_quant.hip, k_norm.hip).
#pragma once

#include "mx.h"
#include "mx_device.h"

namespace svdq {
namespace dev {

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

}  // namespace dev
}  // namespace svdq
