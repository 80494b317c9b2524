// Products of MXFP4 tensors for few rows (decode steps): Y = D(A B^T + bias) and the gated projections, bound by
// reading b once for each 64 rows of A. 16 rows against 8192 x 8192 take 8.0 us (35.7 MB at 4.5 TB/s), one row against
// 24576 x 4096 10.7 us (53.5 MB at 5.0 TB/s), quantised on the way.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 16 rows of A against 16 rows of b, a stage of 128 codes at a
// time; lane (i, g) holds block g of row i of either. A block of waves owns 16 or 32 output columns (gated: the
// gate and up rows of the same 16) and splits K evenly over its waves; every byte of b is used once, so it goes
// straight into registers, a contiguous kilobyte per 16 rows and stage, several stages of requests in flight. The
// waves' partial tiles are added in LDS in a fixed order.
//
// A may be given unquantised: every block then quantises x for itself, which costs vector instructions next to the
// reads of b but no launch. Lane (i, g) loads the 32 elements of its own block and takes their maximum and codes
// without leaving the lane (X_ROWS); for a single row the 16 lanes of a block share it, two elements each, and
// broadcast the code words among them (X_ONE), a quarter of the instructions.
#include "mx.h"
#include "mx_device.h"

namespace svdq {
namespace dev {

enum { A_CODES, X_ROWS, X_ONE };

// Row-of-16 cross-lane moves (DPP): rotation by N lanes, and lane N to all.
template <int N>
__device__ inline u32 row_rotate(u32 v) {
  return (u32)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xF, 0xF, true);
}
template <int N>
__device__ inline u32 row_from(u32 v) {
  return (u32)__builtin_amdgcn_mov_dpp((int)v, 0x150 + N, 0xF, 0xF, true);
}

template <class DT, int MT, int NT, int WAVES, bool GATED, int FORM>
__global__ __launch_bounds__(64 * WAVES) void k_mx_decode(MxGemmParams p) {
  typedef typename DT::T T;
  static_assert(!GATED || NT == 2, "a gate tile and an up tile");
  constexpr bool RAW = FORM != A_CODES;
  constexpr int XW = FORM == X_ONE ? DT::size / 2 : DT::size * 8;  // words of x a lane holds of a stage
  constexpr int BATCH = FORM == X_ROWS ? (DT::size == 4 ? 2 : 4) : (MT >= 2 ? 4 : 8);
  __shared__ float red[WAVES][MT][NT][4][64];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int i = lane & 15, g = lane >> 4;
  // blocks i, i + 8, ... share an XCD: each takes a run of columns, so that the blocks that read the same lines of scale
  // bytes (64 columns' a line) share an L2
  const int run = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  const int n0 = run * (GATED ? 16 : 16 * NT), m0 = blockIdx.y * 16 * MT;
  if (n0 >= p.N) return;
  const int s0 = (int)((int64_t)wave * p.kq / WAVES), s1 = (int)((int64_t)(wave + 1) * p.kq / WAVES);

  const uint8_t *bc[NT], *bs[NT];
#pragma unroll
  for (int n = 0; n < NT; n++) {
    const int64_t col = (int64_t)n0 + i + (GATED ? 0 : 16 * n);
    int64_t row = (col < p.N ? col : p.N - 1) + (GATED && n ? p.N : 0);
    bc[n] = p.b_codes + mx_code_tile_offset(row, p.kq) + g * 16;
    bs[n] = p.b_scales + mx_scale_tiled_index(row, 0, p.kq);
  }
  const uint8_t *ac[MT], *as[MT];
  const T* xr[MT];
#pragma unroll
  for (int m = 0; m < MT; m++) {
    const int64_t row = m0 + 16 * m + i < p.M ? m0 + 16 * m + i : p.M - 1;
    if constexpr (RAW) {
      xr[m] = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    } else {
      ac[m] = p.a_codes + mx_code_tile_offset(row, p.kq) + g * 16;
      as[m] = p.a_scales + mx_scale_tiled_index(row, 0, p.kq);
    }
  }

  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int n = 0; n < NT; n++) acc[m][n] = v4f{0.f, 0.f, 0.f, 0.f};

  struct Step {
    v4i b[NT];
    u32 bsc[NT];
    v4i a[RAW ? 1 : MT];
    u32 asc[RAW ? 1 : MT];
    u32 x[RAW ? MT : 1][RAW ? XW : 1];
  };
  auto load = [&](Step& q, int s) {
#pragma unroll
    for (int n = 0; n < NT; n++) {
      q.b[n] = *reinterpret_cast<const v4i*>(bc[n] + (int64_t)s * 1024);
      q.bsc[n] = *reinterpret_cast<const u32*>(bs[n] + (int64_t)s * 256);
    }
#pragma unroll
    for (int m = 0; m < MT; m++) {
      if constexpr (FORM == X_ONE) {
        const int64_t c = (int64_t)s * 128 + 32 * g + 2 * i;
        if (c + 2 <= p.K) {
          __builtin_memcpy(q.x[m], xr[m] + c, sizeof q.x[m]);
        } else {
#pragma unroll
          for (int k = 0; k < XW; k++) q.x[m][k] = 0;
          if (c < p.K) {
            if constexpr (DT::size == 4)
              q.x[m][0] = __float_as_uint(xr[m][c]);
            else
              q.x[m][0] = xr[m][c];
          }
        }
      } else if constexpr (FORM == X_ROWS) {
        const int64_t c = (int64_t)s * 128 + 32 * g;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const Vec8<DT> v = load8<DT>(xr[m], c + 8 * e, p.K);
#pragma unroll
          for (int k = 0; k < XW / 4; k++) q.x[m][e * (XW / 4) + k] = v.w[k];
        }
      } else {
        q.a[m] = *reinterpret_cast<const v4i*>(ac[m] + (int64_t)s * 1024);
        q.asc[m] = *reinterpret_cast<const u32*>(as[m] + (int64_t)s * 256);
      }
    }
  };
  auto step = [&](const Step& q) {
#pragma unroll
    for (int m = 0; m < MT; m++) {
      v4i a;
      u32 sa;
      if constexpr (FORM == X_ONE) {
        u32 most = amax_bits<DT>(q.x[m]);
        most = max(most, row_rotate<8>(most));
        most = max(most, row_rotate<4>(most));
        most = max(most, row_rotate<2>(most));
        most = max(most, row_rotate<1>(most));
        sa = mx_scale_byte(most);
        u32 w[DT::size * 2] = {};
        w[0] = q.x[m][0];
        if constexpr (DT::size == 4) w[1] = q.x[m][1];
        u32 part = (codes8<DT>(w, sa) & 0xFFu) << (8 * (i & 3));
        part |= (u32)__builtin_amdgcn_mov_dpp((int)part, 0xB1, 0xF, 0xF, true);  // the quad's four bytes
        part |= (u32)__builtin_amdgcn_mov_dpp((int)part, 0x4E, 0xF, 0xF, true);
        a = v4i{(int)row_from<0>(part), (int)row_from<4>(part), (int)row_from<8>(part), (int)row_from<12>(part)};
      } else if constexpr (FORM == X_ROWS) {
        sa = mx_scale_byte(amax_bits<DT>(q.x[m]));
#pragma unroll
        for (int e = 0; e < 4; e++) a[e] = (int)codes8<DT>(q.x[m] + e * (XW / 4), sa);
      } else {
        a = q.a[m];
        sa = q.asc[m] >> (8 * g);
      }
#pragma unroll
      for (int n = 0; n < NT; n++)
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, v8i{q.b[n][0], q.b[n][1], q.b[n][2], q.b[n][3], 0, 0, 0, 0}, acc[m][n],
            4, 4, 0, (int)sa, 0, (int)(q.bsc[n] >> (8 * g)));
    }
  };
  // whole batches, then what is left in halves: a share of K is rarely a multiple of the batch
  int s = s0;
  auto batch = [&](auto n) {
    constexpr int N = decltype(n)::value;
    Step q[N];
#pragma unroll
    for (int u = 0; u < N; u++) load(q[u], s + u);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < N; u++) step(q[u]);
    s += N;
  };
  while (s + BATCH <= s1) batch(std::integral_constant<int, BATCH>());
  if constexpr (BATCH > 4)
    if (s + 4 <= s1) batch(std::integral_constant<int, 4>());
  if constexpr (BATCH > 2)
    if (s + 2 <= s1) batch(std::integral_constant<int, 2>());
  if (s < s1) batch(std::integral_constant<int, 1>());

#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int v = 0; v < 4; v++) red[wave][m][n][v][lane] = acc[m][n][v];
  __syncthreads();
  // entry (m, n, v, lane (i, g)) is row 16 m + 4 g + v of column i of tile n
  constexpr int OUT = MT * (GATED ? 1 : NT) * 256;
  T* y = reinterpret_cast<T*>(p.y);
  for (int e = t; e < OUT; e += 64 * WAVES) {
    const int el = e & 63, v = (e >> 6) & 3, mn = e >> 8;
    const int m = GATED ? mn : mn / NT, n = GATED ? 0 : mn % NT;
    const int64_t row = (int64_t)m0 + 16 * m + 4 * (el >> 4) + v, col = (int64_t)n0 + 16 * n + (el & 15);
    if (row >= p.M || col >= p.N) continue;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; w++) {
      a += red[w][m][n][v][el];
      if (GATED) b += red[w][m][NT - 1][v][el];
    }
    if constexpr (GATED) {
      float h = 0.f;
      with_act(p.act, [&](auto c) { h = act_value<decltype(c)::value, float>(a).a * b; });
      y[row * p.ldy + col] = DT::store(h);
      if (p.gu) {
        T* gu = reinterpret_cast<T*>(p.gu) + row * p.ldgu + col;
        gu[0] = DT::store(a);
        gu[p.N] = DT::store(b);
      }
    } else {
      if (p.bias) a += DT::load(reinterpret_cast<const T*>(p.bias)[col]);
      y[row * p.ldy + col] = DT::store(a);
    }
  }
}

}  // namespace dev

using namespace dev;

// Blocks over N columns, `cols` a block, in whole runs for each XCD.
static int64_t decode_blocks(int64_t N, int64_t cols) { return ((N + cols - 1) / cols + 7) / 8 * 8; }

template <class DT, int MT, int NT, int WAVES, bool GATED, int FORM>
static hipError_t launch_rows(const MxGemmParams& p, hipStream_t stream) {
  const int64_t blocks = decode_blocks(p.N, GATED ? 16 : 16 * NT);
  if (!mx_fits_grid(blocks, 64 * WAVES)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)((p.M + 16 * MT - 1) / (16 * MT)));
  k_mx_decode<DT, MT, NT, WAVES, GATED, FORM><<<grid, 64 * WAVES, 0, stream>>>(p);
  return hipGetLastError();
}

// Column tiles and waves of a block (MxForm: bn = 16 column tiles, waves). A gated block has a gate tile and an up tile.
// Others, by the column tiles there are on 256 compute units; measured at K x N on the GPU's clock, us:
//   up to 256    one tile, eight waves: a block for every compute unit matters most. 8192 x 4096 at one row 5.8, 6.2 with two
//   257 to 512   two tiles, so that a compute unit's blocks are one: 8192 x 5120 at 16 rows 7.7 against 8.7, 8192 x 8192 8.9
//                against 9.7 (1024 x 6000 3.4 both)
//   more         past 16 rows two tiles, so that a's operands serve twice: 8192 x 16384 at 32 rows 17.2, 22.7 with one tile,
//                at 64 rows 23.4 and 34.6. Up to 16 rows, or 32 rows of up to eight stages (1024 x 12288 at 32 rows 4.2,
//                with two tiles 4.4), one tile. Four waves below 64 stages, so that more blocks run at once (1024 x 16384
//                at one row 3.9, 4.5 with eight waves, 4096 x 12288 7.6 and 8.5, 7168 x 12288 10.9 and 11.9); eight from
//                there on, where the waves' own chains of stages count (8192 x 16384 16.4, 21.1 with four, 16384 x 16384
//                28.9 and 31.0, 28672 x 9216 32.0 and 31.8)
MxForm mx_decode_form(int64_t M, int64_t N, int kq, bool gated) {
  const int bm = M <= 16 ? 16 : (M <= 32 ? 32 : 64);
  if (gated) return MxForm{bm, 32, 1, 8};
  const int64_t tiles = (N + 15) / 16;
  if (tiles <= 256) return MxForm{bm, 16, 1, 8};
  if (tiles <= 512 || bm > (kq <= 8 ? 32 : 16)) return MxForm{bm, 32, 1, 8};
  return MxForm{bm, 16, 1, kq < 64 ? 4 : 8};
}

bool mx_decode_fits(int64_t M, int64_t N, int kq, bool gated) {
  const MxForm f = mx_decode_form(M, N, kq, gated);
  return mx_fits_grid(decode_blocks(N, gated ? f.bn / 2 : f.bn), 64 * f.waves);
}

template <class DT, int MT, int FORM>
static hipError_t launch_cols(const MxGemmParams& p, bool gated, hipStream_t stream) {
  if (gated) return launch_rows<DT, MT, 2, 8, true, FORM>(p, stream);
  const MxForm f = mx_decode_form(p.M, p.N, p.kq, false);
  if (f.bn == 32) return launch_rows<DT, MT, 2, 8, false, FORM>(p, stream);
  if constexpr (MT <= 2) {
    if (f.waves == 4) return launch_rows<DT, MT, 1, 4, false, FORM>(p, stream);
  }
  return launch_rows<DT, MT, 1, 8, false, FORM>(p, stream);
}

template <class DT>
static hipError_t launch_decode_t(const MxGemmParams& p, bool gated, hipStream_t stream) {
  if (p.x) return p.M == 1 ? launch_cols<DT, 1, X_ONE>(p, gated, stream) : launch_cols<DT, 1, X_ROWS>(p, gated, stream);
  switch (mx_decode_form(p.M, p.N, p.kq, gated).bm) {
    case 16: return launch_cols<DT, 1, A_CODES>(p, gated, stream);
    case 32: return launch_cols<DT, 2, A_CODES>(p, gated, stream);
    default: return launch_cols<DT, 4, A_CODES>(p, gated, stream);
  }
}

hipError_t launch_mx_decode(const MxGemmParams& p, bool gated, int dtype, hipStream_t stream) {
  switch (dtype) {
    case SVDQ_F32: return launch_decode_t<MxF32>(p, gated, stream);
    case SVDQ_BF16: return launch_decode_t<MxBF16>(p, gated, stream);
    default: return launch_decode_t<MxF16>(p, gated, stream);
  }
}

}  // namespace svdq
