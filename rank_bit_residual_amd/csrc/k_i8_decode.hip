// Products of 8-bit tensors for few rows (decode steps), bound by reading b once for each 64 rows of A.
//
// v_mfma_i32_16x16x64_i8 takes 16 rows of A against 16 rows of b, a stage of 64 codes at a time; lane (i, g) holds codes
// [16 g, 16 g + 16) of row i of either. A block of waves owns 16 NT output columns and splits K evenly over its waves; every byte of
// b is used once, so it goes straight into registers, a contiguous kilobyte per 16 rows and stage, several stages of requests in
// flight. The waves' partial tiles are added in LDS (exact: K is at most 2^17 here). 16 x 8192 x 8192 takes 14.5 us (4.6 TB/s), and one
// unquantised row with b in the last-level cache 12.2 (5.5 TB/s).
//
// A may be given unquantised (RAW): every block then takes the maxima of x's rows for itself and lays its codes in LDS, which costs
// vector instructions next to the reads of b but no launch. Its first reads of b are on their way meanwhile.
#include "i8.h"
#include "i8_device.h"

namespace svdq {
namespace dev {

template <class DT, int MT, int NT, int WAVES, bool RAW>
__global__ __launch_bounds__(64 * WAVES) void k_i8_decode(I8GemmParams p) {
  typedef typename DT::T T;
  constexpr int BATCH = MT * NT >= 4 ? 4 : 8, SLOTS = 4;
  __shared__ int red[WAVES][MT][NT][4][64];
  __shared__ float row_scale[16];
  __shared__ u32 row_max[WAVES][16];
  extern __shared__ __align__(16) uint8_t xcodes[];  // RAW: [M][64 kq]
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int i = lane & 15, g = lane >> 4;
  // blocks i, i + 8, ... share an XCD: each takes a run of columns
  const int run = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  const int64_t n0 = (int64_t)run * 16 * NT;
  const int m0 = blockIdx.y * 16 * MT;
  if (n0 >= p.N) return;
  const int s0 = (int)((int64_t)wave * p.kq / WAVES), s1 = (int)((int64_t)(wave + 1) * p.kq / WAVES);

  const uint8_t* bc[NT];
#pragma unroll
  for (int n = 0; n < NT; n++) {
    const int64_t row = n0 + 16 * n + i;
    bc[n] = p.b_codes + i8_at(row < p.N ? row : p.N - 1, 16 * g, p.kq);
  }
  const uint8_t* ac[MT];
  if constexpr (!RAW) {
#pragma unroll
    for (int m = 0; m < MT; m++) {
      const int row = m0 + 16 * m + i;
      ac[m] = p.a_codes + i8_at(row < p.M ? row : p.M - 1, 16 * g, p.kq);
    }
  }

  v4i acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int n = 0; n < NT; n++) acc[m][n] = v4i{0, 0, 0, 0};

  struct Step {
    v4i b[NT], a[RAW ? 1 : MT];
  };
  auto load = [&](Step& q, int s) {
#pragma unroll
    for (int n = 0; n < NT; n++) q.b[n] = *reinterpret_cast<const v4i*>(bc[n] + (int64_t)s * 1024);
    if constexpr (!RAW) {
#pragma unroll
      for (int m = 0; m < MT; m++) q.a[m] = *reinterpret_cast<const v4i*>(ac[m] + (int64_t)s * 1024);
    }
  };
  // RAW: rows past M repeat the last
  const uint8_t* xrow = xcodes + (int64_t)(i < p.M ? i : p.M - 1) * p.kq * 64 + 16 * g;
  auto step = [&](const Step& q, int s) {
#pragma unroll
    for (int m = 0; m < MT; m++) {
      v4i a;
      if constexpr (RAW)
        a = *reinterpret_cast<const v4i*>(xrow + s * 64);
      else
        a = q.a[m];
#pragma unroll
      for (int n = 0; n < NT; n++) acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, q.b[n], acc[m][n], 0, 0, 0);
    }
  };

  int s = s0;
  Step ahead[RAW ? BATCH : 1];
  if constexpr (RAW) {
    // the first batch of b, requested before x is looked at (a repeated stage is loaded, not used)
#pragma unroll
    for (int u = 0; u < BATCH; u++) load(ahead[u], s0 + u < p.kq ? s0 + u : p.kq - 1);
    __builtin_amdgcn_sched_barrier(0);
    // a wave takes its share of K of every row: in SLOTS vectors a lane, requested together and kept, where they suffice, else row by
    // row and read again
    const T* x = reinterpret_cast<const T*>(p.x);
    const int64_t c0 = (int64_t)s0 * 64 + 8 * lane, c1 = (int64_t)s1 * 64;
    const int per_row = (s1 - s0 + 7) / 8;  // vectors of 512 elements of a row's share
    const bool kept = p.M * per_row <= SLOTS;
    Vec8<DT> v[SLOTS];
    int slot_row[SLOTS];
    int64_t slot_c[SLOTS];
    if (lane < 16) row_max[wave][lane] = 0;
    // lane 0 goes on from what the others wrote
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (kept) {
#pragma unroll
      for (int u = 0; u < SLOTS; u++) {
        slot_row[u] = per_row ? u / per_row : p.M;
        slot_c[u] = c0 + 512 * (per_row ? u % per_row : 0);
        v[u] = zero8<DT>();
        if (slot_row[u] < p.M && slot_c[u] < c1) v[u] = load8<DT>(x + slot_row[u] * p.ldx, slot_c[u], p.K);
      }
#pragma unroll
      for (int u = 0; u < SLOTS; u++) {
        if (slot_row[u] >= p.M) continue;
        const u32 most = wave_umax(amax_bits<DT>(v[u].w));
        if (lane == 0) row_max[wave][slot_row[u]] = max(row_max[wave][slot_row[u]], most);
      }
    } else {
      for (int m = 0; m < p.M; m++) {
        u32 most = 0;
        for (int64_t c = c0; c < c1; c += 512) most = max(most, amax_bits<DT>(load8<DT>(x + m * p.ldx, c, p.K).w));
        most = wave_umax(most);
        if (lane == 0) row_max[wave][m] = most;
      }
    }
    lds_barrier();
    // lane m has row m's scale
    u32 most = 0;
#pragma unroll
    for (int w = 0; w < WAVES; w++) most = max(most, row_max[w][lane & 15]);
    const Scale8 own = scale8(most);
    if (t < 16) row_scale[t] = own.s;
    auto put = [&](int m, int64_t c, const Vec8<DT>& w) {
      const Scale8 q{lane_of(own.s, m), lane_of(own.r, m)};
      float e[8];
#pragma unroll
      for (int k = 0; k < 8; k++) e[k] = elem<DT>(w, k);
      const v2u codes = codes8x8(e, q);
      if (c < c1) *reinterpret_cast<v2u*>(xcodes + (int64_t)m * p.kq * 64 + c) = codes;
    };
    if (kept) {
#pragma unroll
      for (int u = 0; u < SLOTS; u++)
        if (slot_row[u] < p.M) put(slot_row[u], slot_c[u], v[u]);
    } else {
      for (int m = 0; m < p.M; m++)
        for (int64_t c = c0; c - 8 * lane < c1; c += 512) put(m, c, load8<DT>(x + m * p.ldx, c, p.K));
    }
    // a wave reads the codes that it wrote itself
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));  // lgkmcnt(0)
    asm volatile("" ::: "memory");
    const int n = s1 - s0 < BATCH ? s1 - s0 : BATCH;
#pragma unroll
    for (int u = 0; u < BATCH; u++)
      if (u < n) step(ahead[u], s0 + u);
    s += n;
  }
  // whole batches, then what is left in halves: a share of K is rarely a multiple of the batch
  auto batch = [&](auto n) {
    constexpr int N = decltype(n)::value;
    Step q[N];
#pragma unroll
    for (int u = 0; u < N; u++) load(q[u], s + u);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < N; u++) step(q[u], s + u);
    s += N;
  };
  while (s + BATCH <= s1) batch(std::integral_constant<int, BATCH>());
  if constexpr (BATCH > 4)
    if (s + 4 <= s1) batch(std::integral_constant<int, 4>());
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
  T* y = reinterpret_cast<T*>(p.y);
  for (int e = t; e < MT * NT * 256; e += 64 * WAVES) {
    const int el = e & 63, v = (e >> 6) & 3, m = (e >> 8) / NT, n = (e >> 8) % NT;
    const int64_t row = (int64_t)m0 + 16 * m + 4 * (el >> 4) + v, col = n0 + 16 * n + (el & 15);
    if (row >= p.M || col >= p.N) continue;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < WAVES; w++) sum += red[w][m][n][v][el];
    const float sa = RAW ? row_scale[row] : p.a_scales[row];
    const float bz = p.bias ? DT::load(reinterpret_cast<const T*>(p.bias)[col]) : 0.f;
    y[row * p.ldy + col] = DT::store(scaled_far(sum, sa, p.b_scales[col], bz));
  }
}

}  // namespace dev

using namespace dev;

// Blocks over N columns, `cols` a block, in whole runs for each XCD.
static int64_t decode_blocks(int64_t N, int64_t cols) { return ((N + cols - 1) / cols + 7) / 8 * 8; }

constexpr int kRawBytes = 64 * 1024;  // of LDS for the codes of unquantised rows

// One row always; two to four while their shares fit a wave's registers and the columns do not repeat the work too often. As one launch
// against two, us on the GPU's clock (a launch costs 2.7 us of the host's besides): one row x 8192 x 8192 15.7 and 17.4, x 4096 x 4096 6.3 and 7.9,
// x 1024 x 1024 4.2 and 5.1; two rows x 8192 x 4096 11.0 and 11.5; four x 4096 x 4096 7.6 and 8.0, x 1024 x 1024 5.6 and 5.3, x 8192 x 1024 9.5
// and 8.6. (Four x 1024 x 1024 lose 0.3 us on the GPU's clock for the host's 2.7; in a captured graph only the loss counts.)
bool i8_raw_rows(int64_t M, int64_t N, int64_t K, int64_t sc) {
  const int64_t kq = i8_kq(K);
  if (sc != 1 || M * kq * 64 > kRawBytes) return false;
  return M == 1 || (M <= 4 && N <= 8192 && M * ((kq + 63) / 64) <= 4);
}

template <class DT, int MT, int NT, int WAVES, bool RAW>
static hipError_t launch_rows(const I8GemmParams& p, hipStream_t stream) {
  const int64_t blocks = decode_blocks(p.N, 16 * NT);
  if (!mx_fits_grid(blocks, 64 * WAVES)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)((p.M + 16 * MT - 1) / (16 * MT)));
  const unsigned lds = RAW ? (unsigned)(p.M * p.kq * 64) : 0;
  if (RAW && lds > 32 * 1024) {
    // static and dynamic LDS together may pass what a launch has without asking
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_i8_decode<DT, MT, NT, WAVES, RAW>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kRawBytes);
    if (e != hipSuccess) return e;
  }
  k_i8_decode<DT, MT, NT, WAVES, RAW><<<grid, 64 * WAVES, lds, stream>>>(p);
  return hipGetLastError();
}

// The block shape for M x N outputs with the least estimated time in us. A wave's chain is kq / 8 stages; measured (M x K x N): 16 x 4096 x 4096
// with 16 x 16 5.2, 64 x 8192 x 1024 6.6, 128 x 8192 x 1024 with 16 x 32 8.4, 64 x
// 4096 x 4096 with 32 x 32 7.0, 64 x 8192 x 4096 12.0, 256 x 1024 x 1024 3.7, 128 x 4096 x 4096 with 64 x 32 9.3. No less than b's bytes
// from memory, slower with the rows that a block computes: 16 x 8192 x 8192 14.5, 32 x 8192 x 12288 25, 64 x 8192 x 8192 20.
double i8_decode_cost(int64_t M, int64_t N, int kq, MxForm* form) {
  const struct {
    int bm, bn;
    double alone, shared;  // us for a stage of the chain: of one block a unit, of several (each)
  } cand[4] = {{16, 16, 0.29, 0.25}, {16, 32, 0.40, 0.33}, {32, 32, 0.60, 0.50}, {64, 32, 0.89, 1.0}};
  double best = 1e30;
  for (const auto& c : cand) {
    if (c.bm > 16 && c.bm >= 2 * M) continue;
    if ((M + c.bm - 1) / c.bm > 65535) continue;  // the grid's second dimension
    const double b = (double)(((M + c.bm - 1) / c.bm * ((N + c.bn - 1) / c.bn) + 255) / 256), ch = (kq + 7) / 8;
    const double t = 1.9 + 0.5 * b + ch * (c.shared * b > c.alone ? c.shared * b : c.alone);
    const double rows = (double)(M < c.bm ? M : c.bm), again = (double)((M + c.bm - 1) / c.bm - 1);
    const double bytes = 1.5 + (double)N * kq * 64e-6 / 5.8 * (1 + 0.01 * rows) * (1 + 0.3 * again);
    const double least = t > bytes ? t : bytes;
    if (least < best) best = least, *form = MxForm{c.bm, c.bn, 1, 8};
  }
  return best;
}

bool i8_decode_fits(int64_t M, int64_t N, const MxForm& f) {
  return (M + f.bm - 1) / f.bm <= 65535 && mx_fits_grid(decode_blocks(N, f.bn), 64 * f.waves);
}

template <class DT>
static hipError_t launch_decode_t(const I8GemmParams& p, const MxForm& f, hipStream_t stream) {
  if (p.x) return f.bn == 32 ? launch_rows<DT, 1, 2, 8, true>(p, stream) : launch_rows<DT, 1, 1, 8, true>(p, stream);
  if (f.bm == 64) return launch_rows<DT, 4, 2, 8, false>(p, stream);
  if (f.bm == 32) return launch_rows<DT, 2, 2, 8, false>(p, stream);
  return f.bn == 32 ? launch_rows<DT, 1, 2, 8, false>(p, stream) : launch_rows<DT, 1, 1, 8, false>(p, stream);
}

hipError_t launch_i8_decode(const I8GemmParams& p, const MxForm& f, int dtype, hipStream_t stream) {
  switch (dtype) {
    case SVDQ_F32: return launch_decode_t<MxF32>(p, f, stream);
    case SVDQ_BF16: return launch_decode_t<MxBF16>(p, f, stream);
    default: return launch_decode_t<MxF16>(p, f, stream);
  }
}

}  // namespace svdq
