// Products of MXFP4 tensors on gfx950: Y = D(A B^T + bias), and the gated projections
// h = D(act(A Wg^T) * (A Wu^T)) of a feed-forward block.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 K-consecutive E2M1 codes per lane (16 bytes) with the
// lane's own E8M0 byte: exactly one block of an MXFP4 tensor. Products of codes and their scales are
// exact; sums are float32.
//
// Tiles (k_mx_tile): a BM x BN output tile per block of 4 x 2 waves, two per SIMD. K advances in stages of
// 128 codes (64 bytes per row), which land in a ring of four LDS buffers through direct global->LDS
// loads issued two stages ahead; a wave waits on its own loads, one barrier per stage publishes them,
// and a stage's operands are read from LDS under the previous slice's MFMAs. Both operands come in
// 1 KB tiles of 16 rows, one contiguous kilobyte per wave-wide load. LDS rows are 64 bytes; chunk c of row r sits
// at c ^ ((r >> 2) & 3), so that 16 consecutive rows' 16-byte reads meet distinct banks.
// The gated product is the same kernel on a B tile that holds, for each wave, half gate rows and half up rows of
// the same output columns: a lane ends with g and u of its outputs in registers, and the activation and the
// product are its epilogue.
#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "mx.h"
#include "mx_device.h"
#include "tile_store.h"

namespace svdq {
namespace dev {

// ------------------------------------------------------------------------------ tiles
template <int BM, int BN>
struct TileCfg {
  static constexpr int NWV = 8, WN = 2, WM = NWV / WN;
  static constexpr int TM = BM / WM, TN = BN / WN;  // per-wave tile
  static constexpr int MT = TM / 32, NT = TN / 32;
  static constexpr int A_BYTES = BM * 64, B_BYTES = BN * 64;
  static constexpr int A_PER_WAVE = A_BYTES / 1024 / NWV, B_PER_WAVE = B_BYTES / 1024 / NWV;
  static_assert(A_PER_WAVE * NWV * 1024 == A_BYTES && B_PER_WAVE * NWV * 1024 == B_BYTES, "whole wave-wide loads");
  static_assert(TM % 32 == 0 && TN % 64 == 0, "wave tiles are whole MFMA tiles, in gate and up halves");
  static constexpr int SCALE_BYTES = 1024;  // 256 rows x 4 bytes per operand
  static constexpr int STAGE = A_BYTES + B_BYTES + 2 * SCALE_BYTES;
  static constexpr int LPS = A_PER_WAVE + B_PER_WAVE + 1;  // loads per stage and wave
  static constexpr int NS = 4, DIST = 2;                   // ring depth, stages in flight ahead
  static constexpr int SMEM = NS * STAGE;
};

// Block: tile `tid` of tiles_m x tiles_n, stages [s0, s1) of K (an even number, at least two). SPLIT: the
// block's share of K, as float32 sums into its part of p.part; else the finished output.
template <class DT, int BM, int BN, bool GATED, bool SPLIT>
__global__ __launch_bounds__(512) void k_mx_tile(MxGemmParams p) {
  typedef TileCfg<BM, BN> C;
  typedef typename DT::T T;
  constexpr int COLS = GATED ? BN / 2 : BN;  // output columns of a tile
  extern __shared__ __align__(1024) uint8_t smem[];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int l32 = lane & 31, g = lane >> 5;

  // ---- tile order: blocks i, i + 8, ... share an XCD and its L2, so each XCD takes a run of (share of K, tile): few shares,
  // and within one groups of 4 row tiles walked column by column
  const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + COLS - 1) / COLS;
  const int ntiles = tiles_m * tiles_n, all = SPLIT ? ntiles * p.splits : ntiles;
  const int run = (blockIdx.x & 7) * ((all + 7) >> 3) + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= (all + 7) >> 3 || run >= all) return;
  const int split = SPLIT ? run / ntiles : 0, tid = SPLIT ? run - split * ntiles : run;
  const int GM = 4;
  const int group = tid / (GM * tiles_n), gm0 = group * GM;
  const int gsz = (tiles_m - gm0) < GM ? (tiles_m - gm0) : GM;
  const int in_g = tid - group * GM * tiles_n;
  const int m0 = (gm0 + in_g % gsz) * BM, n0 = (in_g / gsz) * COLS;
  int s0 = 0, nst = p.kq;
  if (SPLIT) {
    const int pairs = p.kq / 2;
    s0 = (int)((int64_t)pairs * split / p.splits) * 2;
    nst = (int)((int64_t)pairs * (split + 1) / p.splits) * 2 - s0;
  }

  // row of b behind row rr of the B tile: gated, a wave's columns are half gate rows and half up rows
  auto b_row = [&](int rr) {
    int64_t r;
    if constexpr (GATED) {
      const int w = rr / C::TN, in = rr % C::TN, half = in / (C::TN / 2);
      r = (int64_t)n0 + w * (C::TN / 2) + in % (C::TN / 2) + (half ? p.N : 0);
    } else {
      r = (int64_t)n0 + rr;
    }
    return (int)(r < p.b_rows ? r : p.b_rows - 1);
  };
  auto a_row = [&](int rr) { return m0 + rr < p.M ? m0 + rr : p.M - 1; };

  // ---- sources of this wave's loads: one buffer resource each, based at the 1 KB tile of its first row, so that
  // offsets within it stay below 2 (kq + 1) KB whatever the arrays' sizes; rows past the end repeat the last
  const int64_t a_end = (int64_t)((p.M + 15) >> 4) * p.kq << 10, b_end = (int64_t)((p.b_rows + 15) >> 4) * p.kq << 10;
  const uint8_t *a_base[C::A_PER_WAVE], *b_base[C::B_PER_WAVE];
  int a_rec[C::A_PER_WAVE], b_rec[C::B_PER_WAVE], a_off[C::A_PER_WAVE], b_off[C::B_PER_WAVE];
  const int lr = lane >> 2, chunk = (lane & 3) ^ ((lr >> 2) & 3);
#pragma unroll
  for (int j = 0; j < C::A_PER_WAVE; j++) {
    const int rr = 16 * (wave + C::NWV * j), first = a_row(rr) >> 4, row = a_row(rr + lr);
    const int64_t at = ((int64_t)first * p.kq + s0) << 10;
    a_base[j] = p.a_codes + at;
    a_rec[j] = records(a_end - at);
    a_off[j] = (((row >> 4) - first) * p.kq << 10) + ((row & 15) << 6) + chunk * 16;
  }
#pragma unroll
  for (int j = 0; j < C::B_PER_WAVE; j++) {
    const int rr = 16 * (wave + C::NWV * j), first = b_row(rr) >> 4, row = b_row(rr + lr);
    const int64_t at = ((int64_t)first * p.kq + s0) << 10;
    b_base[j] = p.b_codes + at;
    b_rec[j] = records(b_end - at);
    b_off[j] = (((row >> 4) - first) * p.kq << 10) + ((row & 15) << 6) + chunk * 16;
  }
  // scale words: waves 0-3 load 64 rows of A each, waves 4-7 of B (past the tile: its first rows again)
  const int sw = wave & 3;
  const uint8_t* s_base;
  int s_rec, s_off, s_dst;
  {
    const bool isb = wave >= 4;
    const int rr = 64 * sw < (isb ? BN : BM) ? 64 * sw : 0;
    const int first = (isb ? b_row(rr) : a_row(rr)) >> 6, row = isb ? b_row(rr + lane) : a_row(rr + lane);
    const int64_t at = ((int64_t)first * p.kq + s0) << 8;
    const int64_t end = (int64_t)(((isb ? p.b_rows : p.M) + 63) >> 6) * p.kq << 8;
    s_base = (isb ? p.b_scales : p.a_scales) + at;
    s_rec = records(end - at);
    s_off = (((row >> 6) - first) * p.kq << 8) + ((row & 63) << 2);
    s_dst = C::A_BYTES + C::B_BYTES + (isb ? C::SCALE_BYTES : 0) + sw * 256;
  }

  auto issue = [&](int st) {
    uint8_t* base = smem + (st % C::NS) * C::STAGE;
#pragma unroll
    for (int j = 0; j < C::A_PER_WAVE; j++)
      buffer_to_lds16(a_base[j], a_rec[j], base + (wave + C::NWV * j) * 1024, a_off[j], st * 1024);
#pragma unroll
    for (int j = 0; j < C::B_PER_WAVE; j++)
      buffer_to_lds16(b_base[j], b_rec[j], base + C::A_BYTES + (wave + C::NWV * j) * 1024, b_off[j], st * 1024);
    buffer_to_lds4(s_base, s_rec, base + s_dst, s_off, st * 256);
  };

  v16f acc[C::MT][C::NT];
#pragma unroll
  for (int i = 0; i < C::MT; i++)
#pragma unroll
    for (int j = 0; j < C::NT; j++)
#pragma unroll
      for (int v = 0; v < 16; v++) acc[i][j][v] = 0.f;

  struct Frag {
    v4i a[C::MT], b[C::NT];
  };
  struct Scales {
    u32 a[C::MT], b[C::NT];
  };
  // a 64-code slice's operands: rows 32 apart share the swizzle
  int fa_off[2], fb_off[2];
#pragma unroll
  for (int ks = 0; ks < 2; ks++) {
    fa_off[ks] = lds_swizzle(wm * C::TM + l32, 2 * ks + g);
    fb_off[ks] = C::A_BYTES + lds_swizzle(wn * C::TN + l32, 2 * ks + g);
  }
  const int sa_lane = C::A_BYTES + C::B_BYTES + (wm * C::TM + l32) * 4;
  const int sb_lane = C::A_BYTES + C::B_BYTES + C::SCALE_BYTES + (wn * C::TN + l32) * 4;
  auto read_frag = [&](const uint8_t* base, int ks, Frag& f) {
#pragma unroll
    for (int i = 0; i < C::MT; i++) f.a[i] = *reinterpret_cast<const v4i*>(base + fa_off[ks] + 2048 * i);
#pragma unroll
    for (int j = 0; j < C::NT; j++) f.b[j] = *reinterpret_cast<const v4i*>(base + fb_off[ks] + 2048 * j);
  };
  // a scale word holds a stage's four block bytes; lane (l32, g) uses block 2 ks + g in slice ks: shifted by 8 g
  // once, the MFMA picks byte 2 ks
  const int gsh = 8 * g;
  auto read_scales = [&](const uint8_t* base, Scales& sc) {
#pragma unroll
    for (int i = 0; i < C::MT; i++) sc.a[i] = *reinterpret_cast<const u32*>(base + sa_lane + 128 * i) >> gsh;
#pragma unroll
    for (int j = 0; j < C::NT; j++) sc.b[j] = *reinterpret_cast<const u32*>(base + sb_lane + 128 * j) >> gsh;
  };
  auto mma = [&](const Frag& f, const Scales& sc, auto ks_c) {
    constexpr int KS = decltype(ks_c)::value;
#pragma unroll
    for (int i = 0; i < C::MT; i++)
#pragma unroll
      for (int j = 0; j < C::NT; j++)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            v8i{f.a[i][0], f.a[i][1], f.a[i][2], f.a[i][3], 0, 0, 0, 0},
            v8i{f.b[j][0], f.b[j][1], f.b[j][2], f.b[j][3], 0, 0, 0, 0}, acc[i][j], 4, 4, 2 * KS, (int)sc.a[i], 2 * KS,
            (int)sc.b[j]);
  };
  typedef std::integral_constant<int, 0> Slice0;
  typedef std::integral_constant<int, 1> Slice1;

  // ---- pipeline. Stage s + 2 is issued at the top of iteration s; slice 1 of stage s is read under slice 0's
  // MFMAs; then the wave waits for its own loads of stage s + 1, one barrier publishes every wave's, and stage
  // s + 1's scales and slice 0 are read under slice 1's MFMAs. The same barrier makes refilling buffer
  // (s + 3) % 4 = (s - 1) % 4 safe in iteration s + 1: every wave's reads of stage s - 1 were consumed before it.
  static_assert(C::NS == C::DIST + 2 && C::DIST == 2, "written for two stages in flight");
  constexpr int NR = C::MT + C::NT, NM = C::MT * C::NT;
  constexpr int P1 = NM - 1 < NR ? NM - 1 : NR;
  issue(0);
  issue(1);
  wait_vmcnt<C::LPS>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frag fa, fb, f1;
  Scales sa, sb;
  read_scales(smem, sa);
  read_frag(smem, 0, fa);

  auto stage = [&](int s, Frag& cur0, Scales& scur, Frag& nxt0, Scales& snxt, auto ahead_c) {
    constexpr int AHEAD = decltype(ahead_c)::value;  // stages in flight after s + 1; -1: s is the last
    const uint8_t* base = smem + (s % C::NS) * C::STAGE;
    read_frag(base, 1, f1);
    mma(cur0, scur, Slice0());
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
    for (int q = 0; q < P1; q++) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    if constexpr (NR > P1) __builtin_amdgcn_sched_group_barrier(0x100, NR - P1, 0);
    if constexpr (NM - 1 > P1) __builtin_amdgcn_sched_group_barrier(0x008, NM - 1 - P1, 0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (AHEAD >= 0) {
      wait_vmcnt<C::LPS * AHEAD>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const uint8_t* nb = smem + ((s + 1) % C::NS) * C::STAGE;
      read_scales(nb, snxt);
      read_frag(nb, 0, nxt0);
    }
    mma(f1, scur, Slice1());
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
    for (int q = 0; q < 2 * NR; q++) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (q < NM - 1) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, NM - 1 > 2 * NR ? NM - 1 - 2 * NR : 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  typedef std::integral_constant<int, 1> Steady;
  typedef std::integral_constant<int, 0> LastButOne;
  typedef std::integral_constant<int, -1> Last;
  for (int s = 0; s < nst - 2; s += 2) {
    issue(s + 2);
    stage(s, fa, sa, fb, sb, Steady());
    issue(s + 3);
    stage(s + 1, fb, sb, fa, sa, Steady());
  }
  stage(nst - 2, fa, sa, fb, sb, LastButOne());
  stage(nst - 1, fb, sb, fa, sa, Last());

  // ---- epilogue
  if constexpr (SPLIT) {
    float* part = p.part + (int64_t)split * p.M * p.b_rows;
    if constexpr (GATED) {
      store_tile<MxF32, C, BM, C::NT / 2>(smem, part, p.b_rows, p.M, p.N, m0, n0, wm, wn, lane,
                                          [&](int i, int j, int v) { return acc[i][j][v]; });
      store_tile<MxF32, C, BM, C::NT / 2>(smem, part + p.N, p.b_rows, p.M, p.N, m0, n0, wm, wn, lane,
                                          [&](int i, int j, int v) { return acc[i][j + C::NT / 2][v]; });
    } else {
      store_tile<MxF32, C, BM, C::NT>(smem, part, p.b_rows, p.M, p.N, m0, n0, wm, wn, lane,
                                      [&](int i, int j, int v) { return acc[i][j][v]; });
    }
  } else if constexpr (GATED) {
    T* y = reinterpret_cast<T*>(p.y);
    if (p.gu) {
      T* gu = reinterpret_cast<T*>(p.gu);
      store_tile<DT, C, BM, C::NT / 2>(smem, gu, p.ldgu, p.M, p.N, m0, n0, wm, wn, lane,
                                       [&](int i, int j, int v) { return acc[i][j][v]; });
      store_tile<DT, C, BM, C::NT / 2>(smem, gu + p.N, p.ldgu, p.M, p.N, m0, n0, wm, wn, lane,
                                       [&](int i, int j, int v) { return acc[i][j + C::NT / 2][v]; });
    }
    with_act(p.act, [&](auto c) {
#pragma unroll
      for (int i = 0; i < C::MT; i++)
#pragma unroll
        for (int j = 0; j < C::NT / 2; j++)
#pragma unroll
          for (int v = 0; v < 16; v++)
            acc[i][j][v] = act_value<decltype(c)::value, float>(acc[i][j][v]).a * acc[i][j + C::NT / 2][v];
    });
    store_tile<DT, C, BM, C::NT / 2>(smem, y, p.ldy, p.M, p.N, m0, n0, wm, wn, lane,
                                     [&](int i, int j, int v) { return acc[i][j][v]; });
  } else {
    if (p.bias) {
#pragma unroll
      for (int j = 0; j < C::NT; j++) {
        const int col = n0 + wn * C::TN + 32 * j + l32;
        const float b = DT::load(reinterpret_cast<const T*>(p.bias)[col < p.N ? col : p.N - 1]);
#pragma unroll
        for (int i = 0; i < C::MT; i++)
#pragma unroll
          for (int v = 0; v < 16; v++) acc[i][j][v] += b;
      }
    }
    store_tile<DT, C, BM, C::NT>(smem, reinterpret_cast<T*>(p.y), p.ldy, p.M, p.N, m0, n0, wm, wn, lane,
                                 [&](int i, int j, int v) { return acc[i][j][v]; });
  }
}

// ------------------------------------------------------------------------------ joining split sums
// Adds the parts in order and finishes the outputs, V neighbouring ones per thread (gated: their g and u).
template <class DT, bool GATED, int V>
__global__ __launch_bounds__(256) void k_mx_join(MxGemmParams p) {
  typedef typename DT::T T;
  typedef float vec __attribute__((ext_vector_type(V), aligned(V == 4 ? 16 : 4)));
  const int c = (blockIdx.x * 256 + threadIdx.x) * V;
  if (c >= p.N) return;
  const int64_t stride = (int64_t)p.M * p.b_rows;
  for (int64_t r = blockIdx.y; r < p.M; r += gridDim.y) {
    const float* src = p.part + r * p.b_rows + c;
    vec a = {}, b = {};
    // eight parts requested at a time, added in order (64 x 64 outputs of 64 parts, with the product's kernel: 13.9 us, 16.9 with four)
    for (int s = 0; s < p.splits; s += 8) {
      vec x[8], z[8];
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const int at = s + k < p.splits ? s + k : p.splits - 1;
        x[k] = *reinterpret_cast<const vec*>(src + at * stride);
        if (GATED) z[k] = *reinterpret_cast<const vec*>(src + at * stride + p.N);
      }
#pragma unroll
      for (int k = 0; k < 8; k++) {
        if (s + k >= p.splits) continue;
        a += x[k];
        if (GATED) b += z[k];
      }
    }
    T* y = reinterpret_cast<T*>(p.y) + r * p.ldy + c;
    if constexpr (GATED) {
      if (p.gu) {
        T* gu = reinterpret_cast<T*>(p.gu) + r * p.ldgu + c;
#pragma unroll
        for (int k = 0; k < V; k++) {
          gu[k] = DT::store(a[k]);
          gu[p.N + k] = DT::store(b[k]);
        }
      }
      with_act(p.act, [&](auto act) {
#pragma unroll
        for (int k = 0; k < V; k++) y[k] = DT::store(act_value<decltype(act)::value, float>(a[k]).a * b[k]);
      });
    } else {
#pragma unroll
      for (int k = 0; k < V; k++) y[k] = DT::store(a[k] + (p.bias ? DT::load(reinterpret_cast<const T*>(p.bias)[c + k]) : 0.f));
    }
  }
}

}  // namespace dev

using namespace dev;

// Compute units of the chip: what a plan spreads a product over.
constexpr int kCus = 256;

// How a product is cut: tile shape (bm 0: the kernel for few rows) and shares of K.
struct MxPlan {
  int bm, bn, splits;
};

// The form with the least estimated time in us, from the times measured on this chip (K = 4096 is kq = 32 stages of 128):
//   few rows  (k_mx_decode) b is read again for each 64 rows; with b's elements in millions, up to 32 rows 2.5 us at 1, 3.3
//             to 4 at 17, 7.9 at 67; 64 rows 3.2, 5.2 and 10.1, 128 rows 3.2, 9.0 and 17.8. Small b, many rows, us for each 64
//             of them: 0.29 (1000 columns, K = 512), 0.46 (1000, 1024), 0.79 (1500, 1536), 1.9 (5000, 768).
//             No less than b's bytes from memory: 5.4 TB/s at one row, 9 % slower for every ten rows (143 MB 28 us at one row, 32
//             at 16, 35 at 32, 44 at 64; 570 MB 98, 113, 123 and 160). No less than its blocks: 512 x 82944 7.6 us at one row, 1024 x
//             131072 49 at 64. No less than a wave's stages one after another, 0.25 us each at one row, 0.35 at 16, 0.47 at 32,
//             0.73 at 64 (28672 x 1024: 10.0, 12.7, 16.1, 23.4 us), 0.31 to 0.47 gated at one row
//   128 x 128 two blocks per compute unit; 13 us for up to 256 tiles at kq = 32, 21 for 64 stages, 114 us for 12 tiles a unit
//   128 x 256 one block: 16.5 us for 32 tiles to 21 for 256, 109 us for 1536
//             shares of K run 7 % faster a stage (an XCD's blocks read the same one): 1024 x 65536 x 1024 in 8 shares 48 us, 52 with
//             operands from HBM; 128 x 128 in 4 shares 51 and 62, in 8 shares 51 and 57
//   256 x 256 one block: 23.5 us for 64 tiles, 29 for 192, 35 for 256, 94 for 768; 231 us for 1024 at kq = 64
// A gated product's tiles leave as one to three arrays: 500 x 300 x 2*700 5.4 us, 7.7 with g and u (few rows 5.7 and 6.1); 2048 x 2048 x
// 2*8192 39.9 us on 256 x 256 against 45.4 on 128 x 128.
// Shares of K add the joining launch and the parts' way through memory at 4 TB/s.
// Against few rows, tiles take no less than b's bytes from memory at 5 TB/s, and, for one row, a launch more, as the few-row kernel
// quantises that itself. One row at K x N, the best tiles and the few-row kernel, us: 28672 x 8192 32.6 and 25.3; 16384 x 16384 34.8 and
// 29.4; 65536 x 4096 37.5 and 27.7; 4096 x 128256 55 and 49; 28672 x 1024 13.5 and 10.0; 65536 x 256 12.7 and 14.7.
static MxPlan plan_of(int64_t M, int64_t N, int kq, bool gated) {
  const double b_rows = (double)N * (gated ? 2 : 1), millions = b_rows * kq * 128 * 1e-6, mb = millions * 17 / 32;
  double few = 0.25 * millions + 0.17e-3 * b_rows;
  if (few > 1.6 + 0.11 * millions) few = 1.6 + 0.11 * millions;
  double few_t = M <= 32 ? 2.2 + 0.082 * millions : 3.0 + (double)((M + 63) / 64) * few;
  const double rows = M <= 32 ? (double)M : 64.0;  // past 32 rows a block computes 64
  const double bytes = 2.0 + mb / 5.4 * (1 + 0.009 * rows), blocks = 2.0 + b_rows * (M <= 32 ? 0.08e-3 : 0.36e-3);
  const double in_turn = 2.4 + kq / 8.0 * ((gated ? 0.36 : 0.24) + 0.0075 * rows);
  for (double least : {bytes, blocks, in_turn})
    if (few_t < least) few_t = least;
  MxPlan best{0, 0, 1};
  double best_t = 1e30;
  const int cand[3][2] = {{128, 128}, {128, 256}, {256, 256}};
  for (int c = 0; c < 3; c++) {
    // a 128-wide gated tile reaches its up rows' scales from its gate rows' by a 32-bit offset
    if (gated && c == 0 && N * kq * 4 >= (int64_t)1 << 31) continue;
    const int bm = cand[c][0], cols = gated ? cand[c][1] / 2 : cand[c][1];
    const int64_t tiles = ((M + bm - 1) / bm) * ((N + cols - 1) / cols);
    for (int s = 1; s <= 64; s *= 2) {
      if (s > 1 && (kq / 2 / s < 4 || tiles * s > kCus)) break;
      const double rounds = (double)(tiles * s) / kCus, st = (double)kq / s;
      const double whole = (double)((tiles * s) / kCus), rest = rounds - whole;
      double t;
      if (c == 0)
        t = 4 + 0.29 * st * (rounds > 1 ? rounds : 1);
      else if (c == 1)
        t = (whole + (rest > 0)) * (4 + (s > 1 ? 0.42 : 0.45) * st);
      else
        t = whole * (6 + 0.8 * st) + (rest > 0 ? 6 + st * (0.5 + 0.3 * rest) : 0);
      if (gated && s == 1) t += c == 0 ? 2 : (c == 1 ? 3 : 2) * (whole + (rest > 0));
      if (s > 1) t += 3.0 + (double)M * b_rows * 4 * 2 * s / 4e6;
      if (t < best_t) best = MxPlan{bm, cand[c][1], s}, best_t = t;
    }
  }
  if (M > 64 * 65535) return best;  // past the few-row grid's second dimension
  const double least = 4 + mb / 5.0 + (best.splits > 1 ? 5.0 + (double)M * b_rows * 4 * 2 * best.splits / 4e6 : 0);
  if (best_t < least) best_t = least;
  return few_t <= best_t + (M == 1 ? 2.0 : 0.0) ? MxPlan{0, 0, 1} : best;
}

MxForm mx_product_form(int64_t M, int64_t N, int kq, bool gated) {
  const MxPlan pl = plan_of(M, N, kq, gated);
  return pl.bm ? MxForm{pl.bm, pl.bn, pl.splits, 1} : mx_decode_form(M, N, kq, gated);
}

bool mx_product_decodes(int64_t M, int64_t N, int kq, bool gated) { return plan_of(M, N, kq, gated).bm == 0; }

size_t mx_product_part_bytes(int64_t M, int64_t N, int kq, bool gated) {
  const MxPlan pl = plan_of(M, N, kq, gated);
  return pl.splits > 1 ? (size_t)pl.splits * M * N * (gated ? 2 : 1) * 4 : 0;
}

// Blocks of bm x cols output tiles in `splits` shares of K, in whole runs for each XCD.
static int64_t tile_blocks(int64_t M, int64_t N, int64_t bm, int64_t cols, int64_t splits) {
  return ((M + bm - 1) / bm * ((N + cols - 1) / cols) * splits + 7) / 8 * 8;
}

bool mx_product_fits(int64_t M, int64_t N, int kq, bool gated) {
  const MxPlan pl = plan_of(M, N, kq, gated);
  if (pl.bm == 0) return mx_decode_fits(M, N, kq, gated);
  return mx_fits_grid(tile_blocks(M, N, pl.bm, gated ? pl.bn / 2 : pl.bn, pl.splits), 512);
}

template <class DT, int BM, int BN, bool GATED, bool SPLIT>
static hipError_t launch_tile(const MxGemmParams& p, hipStream_t stream) {
  typedef TileCfg<BM, BN> C;
  const int64_t blocks = tile_blocks(p.M, p.N, BM, GATED ? BN / 2 : BN, p.splits);
  if (!mx_fits_grid(blocks, 64 * C::NWV)) return hipErrorInvalidConfiguration;
  // once per process and device; a second thread at most repeats the same call
  static std::atomic<uint64_t> configured;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(configured.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_mx_tile<DT, BM, BN, GATED, SPLIT>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != hipSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  k_mx_tile<DT, BM, BN, GATED, SPLIT><<<dim3((unsigned)blocks), 512, C::SMEM, stream>>>(p);
  return hipGetLastError();
}

template <class DT, bool GATED>
static hipError_t launch_product_t(const MxGemmParams& p0, const MxPlan& pl, hipStream_t stream) {
  MxGemmParams p = p0;
  p.splits = pl.splits;
  if (p.splits > 1) {
    // the parts are float32 whatever the output's type
    const hipError_t e = pl.bm == 256   ? launch_tile<MxF32, 256, 256, GATED, true>(p, stream)
                         : pl.bn == 256 ? launch_tile<MxF32, 128, 256, GATED, true>(p, stream)
                                        : launch_tile<MxF32, 128, 128, GATED, true>(p, stream);
    if (e != hipSuccess) return e;
    const unsigned rows = p.M < 65535 ? p.M : 65535;
    if (p.N % 4 == 0)
      k_mx_join<DT, GATED, 4><<<dim3((unsigned)((p.N / 4 + 255) / 256), rows), 256, 0, stream>>>(p);
    else
      k_mx_join<DT, GATED, 1><<<dim3((unsigned)((p.N + 255) / 256), rows), 256, 0, stream>>>(p);
    return hipGetLastError();
  }
  return pl.bm == 256   ? launch_tile<DT, 256, 256, GATED, false>(p, stream)
         : pl.bn == 256 ? launch_tile<DT, 128, 256, GATED, false>(p, stream)
                        : launch_tile<DT, 128, 128, GATED, false>(p, stream);
}

hipError_t launch_mx_product(const MxGemmParams& p, bool gated, int dtype, hipStream_t stream) {
  const MxPlan pl = plan_of(p.M, p.N, p.kq, gated);
  if (pl.bm == 0) return launch_mx_decode(p, gated, dtype, stream);
  switch (dtype) {
    case SVDQ_F32: return gated ? launch_product_t<MxF32, true>(p, pl, stream) : launch_product_t<MxF32, false>(p, pl, stream);
    case SVDQ_BF16: return gated ? launch_product_t<MxBF16, true>(p, pl, stream) : launch_product_t<MxBF16, false>(p, pl, stream);
    default: return gated ? launch_product_t<MxF16, true>(p, pl, stream) : launch_product_t<MxF16, false>(p, pl, stream);
  }
}

}  // namespace svdq
