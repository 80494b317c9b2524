// Products of 8-bit tensors on gfx950: y[m, n] = D( (sum_k a[m, k] b[n, k]) sa[m] sb[n] + bias[n] ).
//
// v_mfma_i32_32x32x32_i8 takes 16 K-consecutive codes per lane and sums in int32, so the sum is exact up to K = 2^17
// (2^17 * 127^2 < 2^31); a longer K is cut into shares, whose sums are joined in 64 bits. The scales and the bias enter once, in the
// epilogue: float32 of the sum, times float32(sa sb), plus the bias with one rounding (fma), then the output's own. The same in every form, so an
// output depends on its two rows and its bias alone, not on how many others there are.
//
// Tiles (k_i8_tile): a BM x BN output tile per block of WM x WN waves. K advances in stages of 64 codes (64 bytes per row), which
// land in a ring of LDS buffers through direct global->LDS loads issued DIST stages ahead; a wave waits on its own loads, one
// barrier per stage publishes them, and a stage's operands are read from LDS under the previous slice's MFMAs. Both operands
// come in 1 KB tiles of 16 rows, one contiguous kilobyte per wave-wide load. LDS rows are 64 bytes; chunk c of row r sits at
// c ^ ((r >> 2) & 3), so that 16 consecutive rows' 16-byte reads meet distinct banks.
//
// Bound by the matrix cores and, with the chip full of them, by power: 8192^3 takes 431 us (2.55 POP/s; a loop of nothing but the instruction
// reaches 3.43), 4096 x 4096 x 12288 180. A stage of the 256 x 256 tile takes 1180 cycles, 1024 of them the instructions'; then the epilogue
// 15000 (6000 for the scales, the rest for stores that all units make at once, at the rate of memory).
#include <atomic>
#include <type_traits>

#include "i8.h"
#include "i8_device.h"
#include "tile_store.h"

namespace svdq {
namespace dev {

template <int BM_, int BN_, int WM_, int WN_, int DIST_>
struct I8Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NWV = WM * WN;
  static constexpr int TM = BM / WM, TN = BN / WN;  // per-wave tile
  static constexpr int MT = TM / 32, NT = TN / 32;
  static constexpr int A_BYTES = BM * 64, B_BYTES = BN * 64;
  static constexpr int A_PER_WAVE = A_BYTES / 1024 / NWV, B_PER_WAVE = B_BYTES / 1024 / NWV;
  static_assert(A_PER_WAVE * NWV * 1024 == A_BYTES && B_PER_WAVE * NWV * 1024 == B_BYTES, "whole wave-wide loads");
  static_assert(TM % 32 == 0 && TN % 32 == 0, "wave tiles are whole MFMA tiles");
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int LPS = A_PER_WAVE + B_PER_WAVE;  // loads per stage and wave
  static constexpr int DIST = DIST_, NS = DIST + 2;    // stages in flight ahead, ring depth
  static_assert(DIST % 2 == 0, "the loop takes two stages a turn");
  static constexpr int SMEM = NS * STAGE;
  static constexpr int ALL = SMEM + (BM + BN) * 4;  // behind the ring: the scales of the tile's rows and columns
};

// Blocks i, i + 8, ... share an XCD and its L2, so each XCD takes a run of a product's (share of K, tile): few shares, and within one groups
// of 4 row tiles walked column by column. The place of XCD `xcd`'s block `i` in that order, or -1 past its end.
__device__ inline int run_of(int xcd, int i, int all) {
  const int run = xcd * ((all + 7) >> 3) + i;
  return i >= (all + 7) >> 3 || run >= all ? -1 : run;
}
template <class C>
__device__ inline int tiles_of(const I8GemmParams& p) {
  return ((p.M + C::BM - 1) / C::BM) * ((p.N + C::BN - 1) / C::BN);
}

// Tile `tid` of tiles_m x tiles_n, stages [s0, s0 + nst) of K (an even number, at least two). SPLIT: the block's share of K,
// as int32 sums into its part of p.part; else the finished output.
template <class DT, class C, bool SPLIT>
__device__ __forceinline__ void do_tile(const I8GemmParams& p, int run, uint8_t* smem) {
  typedef typename DT::T T;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int l32 = lane & 31, g = lane >> 5;

  const int tiles_m = (p.M + C::BM - 1) / C::BM, tiles_n = (p.N + C::BN - 1) / C::BN, ntiles = tiles_m * tiles_n;
  const int split = SPLIT ? run / ntiles : 0, tid = SPLIT ? run - split * ntiles : run;
  const int GM = 4;
  const int group = tid / (GM * tiles_n), gm0 = group * GM;
  const int gsz = (tiles_m - gm0) < GM ? (tiles_m - gm0) : GM;
  const int in_g = tid - group * GM * tiles_n;
  const int m0 = (gm0 + in_g % gsz) * C::BM, n0 = (in_g / gsz) * C::BN;
  int s0 = 0, nst = p.kq;
  if (SPLIT) {
    const int pairs = p.kq / 2;
    s0 = (int)((int64_t)pairs * split / p.splits) * 2;
    nst = (int)((int64_t)pairs * (split + 1) / p.splits) * 2 - s0;
  }

  // ---- sources of this wave's loads: one buffer resource each, based at the 1 KB tile of its first row, so that offsets
  // within it stay below 1024 (kq + 1) whatever the arrays' sizes; rows past the end repeat the last
  auto a_row = [&](int rr) { return m0 + rr < p.M ? m0 + rr : p.M - 1; };
  auto b_row = [&](int rr) { return n0 + rr < p.N ? n0 + rr : p.N - 1; };
  const int64_t a_end = (int64_t)((p.M + 15) >> 4) * p.kq << 10, b_end = (int64_t)((p.N + 15) >> 4) * p.kq << 10;
  const uint8_t *a_base[C::A_PER_WAVE], *b_base[C::B_PER_WAVE];
  int a_rec[C::A_PER_WAVE], b_rec[C::B_PER_WAVE], a_off[C::A_PER_WAVE], b_off[C::B_PER_WAVE];
  const int lr = lane >> 2, chunk = (lane & 3) ^ ((lr >> 2) & 3);
#pragma unroll
  for (int j = 0; j < C::A_PER_WAVE; j++) {
    const int rr = 16 * (wave + C::NWV * j);
    const int64_t at = ((int64_t)(a_row(rr) >> 4) * p.kq + s0) << 10;
    a_base[j] = p.a_codes + at;
    a_rec[j] = records(a_end - at);
    a_off[j] = ((a_row(rr + lr) & 15) << 6) + chunk * 16;
  }
#pragma unroll
  for (int j = 0; j < C::B_PER_WAVE; j++) {
    const int rr = 16 * (wave + C::NWV * j);
    const int64_t at = ((int64_t)(b_row(rr) >> 4) * p.kq + s0) << 10;
    b_base[j] = p.b_codes + at;
    b_rec[j] = records(b_end - at);
    b_off[j] = ((b_row(rr + lr) & 15) << 6) + chunk * 16;
  }
  if constexpr (!SPLIT) {
    // 64 scales a load; they are older than any stage's loads, so the first stage's wait covers them
    for (int q = wave; q < (C::BM + C::BN) / 64; q += C::NWV) {
      const bool isb = q >= C::BM / 64;
      const int first = isb ? n0 : m0, row = isb ? b_row(64 * q - C::BM + lane) : a_row(64 * q + lane);
      const float* src = (isb ? p.b_scales : p.a_scales) + first;
      buffer_to_lds4(reinterpret_cast<const uint8_t*>(src), records((int64_t)((isb ? p.N : p.M) - first) * 4), smem + C::SMEM + q * 256,
                     (row - first) * 4, 0);
    }
  }
  auto issue = [&](int st) {
    uint8_t* base = smem + (st % C::NS) * C::STAGE;
#pragma unroll
    for (int j = 0; j < C::A_PER_WAVE; j++)
      buffer_to_lds16(a_base[j], a_rec[j], base + (wave + C::NWV * j) * 1024, a_off[j], st * 1024);
#pragma unroll
    for (int j = 0; j < C::B_PER_WAVE; j++)
      buffer_to_lds16(b_base[j], b_rec[j], base + C::A_BYTES + (wave + C::NWV * j) * 1024, b_off[j], st * 1024);
  };

  v16i acc[C::MT][C::NT];
#pragma unroll
  for (int i = 0; i < C::MT; i++)
#pragma unroll
    for (int j = 0; j < C::NT; j++)
#pragma unroll
      for (int v = 0; v < 16; v++) acc[i][j][v] = 0;

  struct Frag {
    v4i a[C::MT], b[C::NT];
  };
  // a 32-code slice's operands: rows 32 apart share the swizzle
  int fa_off[2], fb_off[2];
#pragma unroll
  for (int ks = 0; ks < 2; ks++) {
    fa_off[ks] = lds_swizzle(wm * C::TM + l32, 2 * ks + g);
    fb_off[ks] = C::A_BYTES + lds_swizzle(wn * C::TN + l32, 2 * ks + g);
  }
  auto read_frag = [&](const uint8_t* base, int ks, Frag& f) {
#pragma unroll
    for (int i = 0; i < C::MT; i++) f.a[i] = *reinterpret_cast<const v4i*>(base + fa_off[ks] + 2048 * i);
#pragma unroll
    for (int j = 0; j < C::NT; j++) f.b[j] = *reinterpret_cast<const v4i*>(base + fb_off[ks] + 2048 * j);
  };
  auto mma = [&](const Frag& f) {
#pragma unroll
    for (int i = 0; i < C::MT; i++)
#pragma unroll
      for (int j = 0; j < C::NT; j++) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
  };

  // ---- pipeline. Stage s + DIST is issued at the top of iteration s; slice 1 of stage s is read under slice 0's MFMAs; then the
  // wave waits for its own loads of stage s + 1, one barrier publishes every wave's, and stage s + 1's slice 0 is read under slice
  // 1's MFMAs. The same barrier makes refilling buffer (s + 1 + DIST) % NS = (s - 1) % NS safe in iteration s + 1: every
  // wave's reads of stage s - 1 were consumed before it.
  constexpr int NR = C::MT + C::NT, NM = C::MT * C::NT;
  constexpr int P1 = NM - 1 < NR ? NM - 1 : NR;
  float sb[C::NT], bz[C::NT];  // the lane's columns: scales and bias, on hand before the loop
  if constexpr (!SPLIT) {
#pragma unroll
    for (int j = 0; j < C::NT; j++)
      bz[j] = p.bias ? DT::load(reinterpret_cast<const T*>(p.bias)[b_row(wn * C::TN + 32 * j + l32)]) : 0.f;
  }
  const int first = nst < C::DIST ? nst : C::DIST;
  for (int s = 0; s < first; s++) issue(s);
  wait_stage_upto<C::LPS, C::DIST - 1>(first - 1);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  const float* scales = reinterpret_cast<const float*>(smem + C::SMEM);
  bool far = false;
  if constexpr (!SPLIT) {
#pragma unroll
    for (int j = 0; j < C::NT; j++) {
      sb[j] = scales[C::BM + wn * C::TN + 32 * j + l32];
      asm volatile("" : "+v"(sb[j]), "+v"(bz[j]));
    }
    // one scale a lane: whether any of the wave's rows and columns is far
    far = !tame(scales[wm * C::TM + lane % C::TM]);
#pragma unroll
    for (int j = 0; j < C::NT; j++) far |= !tame(sb[j]);
    static_assert(C::TM <= 64, "a wave's rows fit its lanes");
    far = __builtin_amdgcn_ballot_w64(far) != 0;
  }
  Frag fa, fb, f1;
  read_frag(smem, 0, fa);

  // `ahead`: stages issued after s + 1 (a constant in the steady state), or -1: s is the last
  auto stage = [&](int s, Frag& cur0, Frag& nxt0, auto ahead) {
    const uint8_t* base = smem + (s % C::NS) * C::STAGE;
    read_frag(base, 1, f1);
    mma(cur0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
    for (int q = 0; q < P1; q++) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    if constexpr (NR > P1) __builtin_amdgcn_sched_group_barrier(0x100, NR - P1, 0);
    if constexpr (NM - 1 > P1) __builtin_amdgcn_sched_group_barrier(0x008, NM - 1 - P1, 0);
    __builtin_amdgcn_sched_barrier(0);
    constexpr bool steady = !std::is_same<decltype(ahead), int>::value;
    if (steady || ahead >= 0) {
      if constexpr (steady)
        wait_vmcnt<C::LPS * decltype(ahead)::value>();
      else
        wait_stage_upto<C::LPS, C::DIST - 1>(ahead);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      read_frag(smem + ((s + 1) % C::NS) * C::STAGE, 0, nxt0);
    }
    mma(f1);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
    for (int q = 0; q < NR; q++) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (q < NM - 1) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, NM - 1 > NR ? NM - 1 - NR : 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  typedef std::integral_constant<int, C::DIST - 1> Steady;
  int s = 0;
  for (; s < nst - C::DIST; s += 2) {
    issue(s + C::DIST);
    stage(s, fa, fb, Steady());
    issue(s + 1 + C::DIST);
    stage(s + 1, fb, fa, Steady());
  }
  for (; s < nst; s += 2) {
    stage(s, fa, fb, nst - 2 - s);
    stage(s + 1, fb, fa, nst - 3 - s);
  }

  // ---- epilogue
  if constexpr (SPLIT) {
    store_tile<MxF32, C, C::BM, C::NT>(smem, reinterpret_cast<float*>(p.part) + (int64_t)split * p.M * p.N, p.N, p.M, p.N, m0, n0,
                                       wm, wn, lane, [&](int i, int j, int v) { return __int_as_float(acc[i][j][v]); });
  } else {
#pragma unroll
    for (int i = 0; i < C::MT; i++) {
      // entry v of the lane lies in row 8 (v / 4) + 4 g + v % 4
      v4f sa[4];
      bool any = far;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        sa[q] = *reinterpret_cast<const v4f*>(scales + wm * C::TM + 32 * i + 8 * q + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; e++) any |= !tame(sa[q][e]);
      }
      if (__builtin_amdgcn_ballot_w64(any)) {
#pragma unroll
        for (int j = 0; j < C::NT; j++)
#pragma unroll
          for (int v = 0; v < 16; v++) {
            acc[i][j][v] = __float_as_int(scaled_far(acc[i][j][v], sa[v >> 2][v & 3], sb[j], bz[j]));
            __builtin_amdgcn_sched_barrier(0);  // rarely taken: one at a time, in few registers
          }
      } else {
#pragma unroll
        for (int j = 0; j < C::NT; j++)
#pragma unroll
          for (int v = 0; v < 16; v++)
            acc[i][j][v] = __float_as_int(scaled(acc[i][j][v], sa[v >> 2][v & 3], sb[j], bz[j]));
      }
    }
    store_tile<DT, C, C::BM, C::NT>(smem, reinterpret_cast<T*>(p.y), p.ldy, p.M, p.N, m0, n0, wm, wn, lane,
                                    [&](int i, int j, int v) { return __int_as_float(acc[i][j][v]); });
  }
}

template <class DT, class C, bool SPLIT>
__global__ __launch_bounds__(64 * C::NWV) void k_i8_tile(I8GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int run = run_of(blockIdx.x & 7, blockIdx.x >> 3, SPLIT ? tiles_of<C>(p) * p.splits : tiles_of<C>(p));
  if (run >= 0) do_tile<DT, C, SPLIT>(p, run, smem);
}

// Two products that do not wait for each other in one launch, the one with the longer tiles first: the second's fill the units that the
// first's leave, and a launch less waits for the one before it (measured beside pair_time).
template <class DT, class C>
__global__ __launch_bounds__(64 * C::NWV) void k_i8_tile2(I8GemmParams p0, I8GemmParams p1) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int n0 = tiles_of<C>(p0), i = blockIdx.x >> 3, per0 = (n0 + 7) >> 3;
  const bool second = i >= per0;
  I8GemmParams p = p0;
  if (second) p = p1;
  const int run = run_of(blockIdx.x & 7, second ? i - per0 : i, second ? tiles_of<C>(p1) : n0);
  if (run >= 0) do_tile<DT, C, false>(p, run, smem);
}

// ------------------------------------------------------------------------------ joining split sums
// Adds the parts in 64 bits and finishes the outputs, V neighbouring ones per thread. Bound by reading them: eight parts are requested at a
// time.
template <class DT, int V>
__global__ __launch_bounds__(256) void k_i8_join(I8GemmParams p) {
  typedef typename DT::T T;
  typedef int vec __attribute__((ext_vector_type(V), aligned(V == 4 ? 16 : 4)));
  const int c = (blockIdx.x * 256 + threadIdx.x) * V;
  if (c >= p.N) return;
  const int64_t stride = (int64_t)p.M * p.N;
  float sb[V], bz[V];
#pragma unroll
  for (int k = 0; k < V; k++) {
    sb[k] = p.b_scales[c + k];
    bz[k] = p.bias ? DT::load(reinterpret_cast<const T*>(p.bias)[c + k]) : 0.f;
  }
  for (int64_t r = blockIdx.y; r < p.M; r += gridDim.y) {
    const int* src = p.part + r * p.N + c;
    const float sa = p.a_scales[r];
    int64_t sum[V] = {};
    for (int s = 0; s < p.splits; s += 8) {
      vec x[8];
#pragma unroll
      for (int k = 0; k < 8; k++) x[k] = *reinterpret_cast<const vec*>(src + (s + k < p.splits ? s + k : p.splits - 1) * stride);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        if (s + k >= p.splits) continue;
#pragma unroll
        for (int e = 0; e < V; e++) sum[e] += x[k][e];
      }
    }
    T* y = reinterpret_cast<T*>(p.y) + r * p.ldy + c;
#pragma unroll
    for (int k = 0; k < V; k++) y[k] = DT::store(scaled_long(sum[k], sa, sb[k], bz[k]));
  }
}

}  // namespace dev

using namespace dev;

// Compute units of the chip: what a plan spreads a product over. Stages whose int32 sums cannot overflow: 2^17 codes.
constexpr int kCus = 256, kExactStages = 2048;
constexpr double kLaunch = 2.0;  // us that a launch of its own costs the second of two products

typedef I8Cfg<64, 64, 2, 2, 4> Tile64;
typedef I8Cfg<64, 128, 2, 2, 4> Tile64n;
typedef I8Cfg<128, 128, 4, 2, 2> Tile128;
typedef I8Cfg<256, 256, 4, 2, 2> Tile256;

// The form with the least estimated time in us, from the times measured on this chip (M x K x N, us; K = 4096 is 64 stages of 64):
//   64 x 64    three blocks a compute unit (b: blocks for each): 2048 x 2048 x 512 (b 1) 8.7, 512 x 4096 x 4096 (2) 16.8, 4096^3 (16) 110,
//              4096 x 512 x 4096 (16) 27
//   64 x 128   two: 512 x 4096 x 4096 (1) 15.2, 1000 x 4096 x 4096 (2) 26, 4096^3 (8) 89, 4096 x 512 x 4096 (8) 25
//   128 x 128  two: 1000 x 4096 x 4096 (1) 22.3, 2048 x 4096 x 4096 (2) 37, 4096^3 (4) 71, 4096 x 512 x 4096 (4) 26
//   256 x 256  one: 1024 x 4096 x 4096 (64 blocks) 41, 1000 x 4096 x 11000 (172) 52, 4096^3 (256) 62, 4096 x 512 x 4096 (256) 19.6,
//              8192^3 (1024) 431
// Operands past the last-level cache cost the smaller tiles a quarter more, as they read them more often: 1024 x 65536 x 1024 in four
// shares of 128 x 128 105, in 16 of 256 x 256 81. Shares of K add the joining launch and the parts' way through memory.
// The kernel for few rows has its own estimate (i8_decode_cost).
struct Cost {
  int bm, bn;
  double first, alone, shared, out;  // us: a block's own, a stage of one block a unit, of several (each), a further block's epilogue
};
static const Cost kForms[4] = {{64, 64, 3.5, 0.15, 0.095, 0.65}, {64, 128, 4.0, 0.17, 0.16, 1.6}, {128, 128, 4.5, 0.265, 0.21, 3.0}, {256, 256, 0, 0, 0, 0}};

static double tile_time(const Cost& c, int64_t M, int64_t N, int kq, int s) {
  const double least = 3.5 + ((double)M + (double)N) * kq * 64e-6 / 5.0;  // the operands' bytes from memory
  const double cold = ((double)M + (double)N) * kq * 64 > 64e6 ? 1.25 : 1.0;
  const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
  const double st = (double)kq / s;
  double t;
  if (c.bm == 256) {
    const double whole = (double)((tiles * s) / kCus), rest = (double)(tiles * s) / kCus - whole;
    t = whole * (10.8 + 0.764 * st) + (rest > 0 ? 4 + 7 * rest + st * (0.52 + 0.22 * rest) : 0);
  } else {
    const double b = (double)((tiles * s + kCus - 1) / kCus);
    const double rate = b <= 1 ? c.alone : (c.shared * b > c.alone + c.shared * 0.6 ? c.shared * b : c.alone + c.shared * 0.6);
    t = c.first + st * rate * cold + (b > 1 ? c.out * (b - 1) : 0);
  }
  if (t < least) t = least;
  if (M == 1) t += 2.0;  // the launch that quantises a row, which the other kernel does itself
  if (s > 1) t += 3.0 + (double)M * N * 4 * 2 * s / 5.5e6;
  return t;
}

static MxForm choose(int64_t M, int64_t N, int kq, double& best_t) {
  MxForm best{0, 0, 1, 1};
  best_t = 1e30;
  if (kq <= kExactStages) best_t = i8_decode_cost(M, N, kq, &best);
  for (const Cost& c : kForms) {
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (int s = 1; s <= kq / 2; s *= 2) {
      if ((kq / 2 + s - 1) / s * 2 > kExactStages) continue;
      if (s > 1 && best_t < 1e30 && (kq / 2 / s < 4 || tiles * s > 2 * kCus)) break;
      const double t = tile_time(c, M, N, kq, s);
      if (t < best_t) best = MxForm{c.bm, c.bn, s, 1}, best_t = t;
    }
  }
  return best;
}

// (A call asks several times for the sizes that it was given; a backward pass has two of them.)
static MxForm plan_of(int64_t M, int64_t N, int kq, double* time = nullptr) {
  struct Plan {
    int64_t M, N;
    int kq;
    MxForm f;
    double t;
  };
  static thread_local Plan last[2] = {};
  static thread_local int older = 0;
  auto is = [&](const Plan& p) { return p.M == M && p.N == N && p.kq == kq; };
  const int at = is(last[0]) ? 0 : (is(last[1]) ? 1 : older);
  Plan& p = last[at];
  if (!is(p)) p.f = choose(M, N, kq, p.t), p.M = M, p.N = N, p.kq = kq, older = 1 - at;
  if (time) *time = p.t;
  return p.f;
}

MxForm i8_product_form(int64_t M, int64_t N, int kq) { return plan_of(M, N, kq); }

size_t i8_product_part_bytes(int64_t M, int64_t N, int kq) {
  const MxForm f = plan_of(M, N, kq);
  return f.splits > 1 ? (size_t)f.splits * M * N * 4 : 0;
}

// Blocks of output tiles in `splits` shares of K, in whole runs for each XCD.
static int64_t tile_blocks(int64_t M, int64_t N, const MxForm& f) {
  return ((M + f.bm - 1) / f.bm * ((N + f.bn - 1) / f.bn) * f.splits + 7) / 8 * 8;
}

bool i8_product_fits(int64_t M, int64_t N, int kq) {
  const MxForm f = plan_of(M, N, kq);
  return f.waves > 1 ? i8_decode_fits(M, N, f) : mx_fits_grid(tile_blocks(M, N, f), 512);
}

// Lets `kernel` have the LDS of C: once per process and device; a second thread at most repeats the same call.
template <class C>
static hipError_t configure(const void* kernel, std::atomic<uint64_t>& configured) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(configured.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, C::ALL);
    if (e == hipSuccess) configured.fetch_or(bit, std::memory_order_relaxed);
  }
  return e;
}

template <class DT, class C, bool SPLIT>
static hipError_t launch_tile(const I8GemmParams& p, const MxForm& f, hipStream_t stream) {
  const int64_t blocks = tile_blocks(p.M, p.N, f);
  if (!mx_fits_grid(blocks, 64 * C::NWV)) return hipErrorInvalidConfiguration;
  static std::atomic<uint64_t> configured;
  const hipError_t e = configure<C>(reinterpret_cast<const void*>(&k_i8_tile<DT, C, SPLIT>), configured);
  if (e != hipSuccess) return e;
  k_i8_tile<DT, C, SPLIT><<<dim3((unsigned)blocks), 64 * C::NWV, C::ALL, stream>>>(p);
  return hipGetLastError();
}

template <class DT, class C>
static hipError_t launch_tile2(const I8GemmParams& p, const I8GemmParams& q, const MxForm& f, hipStream_t stream) {
  static std::atomic<uint64_t> configured;
  const hipError_t e = configure<C>(reinterpret_cast<const void*>(&k_i8_tile2<DT, C>), configured);
  if (e != hipSuccess) return e;
  const int64_t blocks = tile_blocks(p.M, p.N, f) + tile_blocks(q.M, q.N, f);
  k_i8_tile2<DT, C><<<dim3((unsigned)blocks), 64 * C::NWV, C::ALL, stream>>>(p, q);
  return hipGetLastError();
}

template <class DT, bool SPLIT>
static hipError_t launch_form(const I8GemmParams& p, const MxForm& f, hipStream_t stream) {
  if (f.bm == 64 && f.bn == 64) return launch_tile<DT, Tile64, SPLIT>(p, f, stream);
  if (f.bm == 64) return launch_tile<DT, Tile64n, SPLIT>(p, f, stream);
  if (f.bm == 256) return launch_tile<DT, Tile256, SPLIT>(p, f, stream);
  return launch_tile<DT, Tile128, SPLIT>(p, f, stream);
}

template <class DT>
static hipError_t launch_product_t(const I8GemmParams& p0, const MxForm& f, hipStream_t stream) {
  I8GemmParams p = p0;
  p.splits = f.splits;
  if (p.splits == 1) return launch_form<DT, false>(p, f, stream);
  // the parts are int32 whatever the output's type
  const hipError_t e = launch_form<MxF32, true>(p, f, stream);
  if (e != hipSuccess) return e;
  const unsigned rows = p.M < 65535 ? p.M : 65535;
  if (p.N % 4 == 0)
    k_i8_join<DT, 4><<<dim3((unsigned)((p.N / 4 + 255) / 256), rows), 256, 0, stream>>>(p);
  else
    k_i8_join<DT, 1><<<dim3((unsigned)((p.N + 255) / 256), rows), 256, 0, stream>>>(p);
  return hipGetLastError();
}

// Two products in one launch with tiles of one form, us: the stages that a unit gets of both, or the longest block alone. Measured (M x K x N of
// y; dx and dw in 64 x 64, 64 x 128, 128 x 128, 256 x 256 tiles, and in two launches): 512 x 512 x 2048 9.1, 9.9, 12.2, 24.8, 13.8; 515 x 1440 x 2731 15.1,
// 14.6, 17.5, 31.2, 19.6; 1024 x 4096 x 1024 22.2, 20.0, 16.0, 19.5, 19.9; 2048 x 4096 x 4096 111, 95, 75, 66, 76; 4096 x 4096 x 12288 256 x 256
// 339, two launches 348. Where dw is much larger than dx the stores count and two launches stay: 16 x 4096 x 12288 61, 60, 71, 112 and 47.
static double pair_time(const Cost& c, int64_t M0, int64_t N0, int kq0, int64_t M1, int64_t N1, int kq1) {
  const double tiles0 = (double)((M0 + c.bm - 1) / c.bm) * (double)((N0 + c.bn - 1) / c.bn);
  const double tiles1 = (double)((M1 + c.bm - 1) / c.bm) * (double)((N1 + c.bn - 1) / c.bn);
  const double b = (tiles0 + tiles1) / kCus, stages = (tiles0 * kq0 + tiles1 * kq1) / kCus, longest = kq0 > kq1 ? kq0 : kq1;
  if (c.bm == 256) {
    const double full = b < 1 ? b : 1, all = 10.8 * b + 0.764 * stages, one = 4 + 7 * full + longest * (0.52 + 0.22 * full);
    return all > one ? all : one;
  }
  const double cold = (((double)M0 + (double)N0) * kq0 + ((double)M1 + (double)N1) * kq1) * 64 > 64e6 ? 1.25 : 1.0;
  const double all = c.first + stages * c.shared * cold + (b > 1 ? c.out * (b - 1) : 0), one = c.first + longest * c.alone * cold;
  const double crowd = c.bn == 64 ? 1.1 : 1.0;  // of the smallest tiles' stores
  return (all > one ? all : one) * crowd;
}

// The form that two products share in one launch, or none (bm 0): the one of the least time, if that is less than two launches'.
MxForm i8_pair_form(int64_t M0, int64_t N0, int kq0, int64_t M1, int64_t N1, int kq1) {
  MxForm best{0, 0, 1, 1};
  if (kq0 > kExactStages || kq1 > kExactStages) return best;
  double t0, t1;
  plan_of(M0, N0, kq0, &t0);
  plan_of(M1, N1, kq1, &t1);
  double best_t = t0 + t1 + kLaunch;
  for (const Cost& c : kForms) {
    const MxForm f{c.bm, c.bn, 1, 1};
    const double t = pair_time(c, M0, N0, kq0, M1, N1, kq1);
    if (t < best_t && mx_fits_grid(tile_blocks(M0, N0, f) + tile_blocks(M1, N1, f), 512)) best = f, best_t = t;
  }
  return best;
}

template <class DT>
static hipError_t launch_pair(const I8GemmParams& p, const I8GemmParams& q, const MxForm& f, hipStream_t stream) {
  if (f.bm == 64 && f.bn == 64) return launch_tile2<DT, Tile64>(p, q, f, stream);
  if (f.bm == 64) return launch_tile2<DT, Tile64n>(p, q, f, stream);
  if (f.bm == 256) return launch_tile2<DT, Tile256>(p, q, f, stream);
  return launch_tile2<DT, Tile128>(p, q, f, stream);
}

hipError_t launch_i8_products(const I8GemmParams& p, const I8GemmParams& q, int dtype, hipStream_t stream) {
  if (q.kq > p.kq) return launch_i8_products(q, p, dtype, stream);
  const MxForm f = i8_pair_form(p.M, p.N, p.kq, q.M, q.N, q.kq);
  if (!f.bm) {
    const hipError_t e = launch_i8_product(p, dtype, stream);
    return e != hipSuccess ? e : launch_i8_product(q, dtype, stream);
  }
  switch (dtype) {
    case SVDQ_F32: return launch_pair<MxF32>(p, q, f, stream);
    case SVDQ_BF16: return launch_pair<MxBF16>(p, q, f, stream);
    default: return launch_pair<MxF16>(p, q, f, stream);
  }
}

hipError_t launch_i8_product(const I8GemmParams& p, int dtype, hipStream_t stream) {
  const MxForm f = plan_of(p.M, p.N, p.kq);
  if (f.waves > 1) return launch_i8_decode(p, f, dtype, stream);
  switch (dtype) {
    case SVDQ_F32: return launch_product_t<MxF32>(p, f, stream);
    case SVDQ_BF16: return launch_product_t<MxBF16>(p, f, stream);
    default: return launch_product_t<MxF16>(p, f, stream);
  }
}

}  // namespace svdq
