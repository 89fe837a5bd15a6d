// Low-rank adapters of many requests beside a projection that they share, for gfx950:
//
//   out[i] = RNE(base[i] + scale[a] * (x[i] . down[a]^T) . up[a]^T),   a = index[i]
//
// over rows whose requests use different adapters, or none (index -1: out[i] = base[i]).  The inner
// dimension, the rank, is small, so the products are bound by the bytes of x, base and out
// (and, for few rows, of the adapters); both run on the matrix cores.
//   k_lowrank_down  t = x . down^T: 16 or 32 rows a tile, against the columns of the adapters that
//                   its rows use, each once; K in parts where rows are few.  Sums in float32.
//   k_lowrank_up    out = base + t . up^T: a tile goes through the adapters of its rows one after the
//                   other, and each row takes the one that is its own.  Sums of different adapters do
//                   not meet, so an infinity or NaN in one adapter stays out of the other requests' rows.
// t, scaled, enters the second product as the sum of two 16-bit values, hi and lo = RNE16(t - hi): rounded once
// it would cost the output up to 2^-9 of the adapter's part in bfloat16, in two pieces 2^-16 (fp16
// 2^-22), for a second matrix instruction in a kernel that waits for memory.  A float32 output of bfloat16 operands
// would show 2^-16: it takes a third piece, and nothing is lost.  hi is cut off, so that lo has t's
// sign, and neither is zero where t is not: an infinity in up times t is then the infinity that the
// formula gives, and not NaN.  (Taking NaN sums from hi alone costs the inner loop 84 -> 93 us, rank 128 159 ->
// 196.)  An fp16 row is scaled by the power of two that brings its largest |t| to [2^13, 2^14), since t is not
// bound to fp16's range; the products are scaled back, both exactly (a lo below 2^-24 is lost).
//
// Measured, three sets of buffers in turn: 17776 rows of seven requests, 1920 -> 5760, rank 32, 32 + 85 us (base
// and out alone are 79 us at a large copy's rate, and take 78 in a copy with this access pattern), rank 64
// 43 + 108, rank 128 73 + 163: there every tile's reads of up and down through the second-level caches bound
// both; with base and out in float32 32 + 154, 42 + 171 and 74 + 223; 48 requests of one row over 12 adapters, 4096 ->
// 12288, rank 16, 5.8 + 8.9 us; one row, 1920 -> 5760, rank 64, 6.5 + 4.8 us: launches and dependent loads.  Tried and not kept: loads of base or stores of out past the
// cache (109 -> 113 to 123 us), several column tiles of a workgroup one after the other (94 -> 111 in a plain
// copy), a contiguous range of tiles for each XCD (92 -> 105), tiles of 64 rows.
#include <algorithm>
#include <type_traits>

#include "dev_common.h"
#include "gemm_common.h"
#include "rows_common.h"
#include "vq_internal.h"

namespace vqk {

struct LowrankArgs {
  const uint16_t* x;
  const uint16_t* down;  // [adapters, rank, k]
  const uint16_t* up;    // [adapters, n, rank]
  const int32_t* index;
  const float* scale;  // or nullptr
  const void* base;
  void* out;
  float* t;  // [splits, rows, rank], of lowrank_t_rows rows in all
  int64_t ldx, ldb, ldo, rows;
  int adapters, rank, k, n, splits, chunks, col_tiles;
};

template <int DT>
struct Half {
  typedef typename std::conditional<DT == DT_BF16, __bf16, _Float16>::type T;
  typedef T V8 __attribute__((ext_vector_type(8)));
};
template <int DT>
__device__ __forceinline__ v4f mfma32(typename Half<DT>::V8 a, typename Half<DT>::V8 b, v4f c) {
  if constexpr (DT == DT_BF16) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The adapter of row i, -1 for none.
__device__ __forceinline__ int adapter_of(const LowrankArgs& g, int64_t i) {
  const int a = i < g.rows ? g.index[i] : -1;
  return a >= 0 && a < g.adapters ? a : -1;
}
// The different adapters among the lanes' (a >= 0): lane d gets the d-th in `list`; returns their number.
__device__ __forceinline__ int distinct(int a, int& list) {
  const int lane = threadIdx.x & 63;
  uint64_t left = __ballot(a >= 0);
  int n = 0;
  list = -1;
  while (left) {
    const int v = __builtin_amdgcn_readlane(a, __builtin_ctzll(left));
    left &= ~__ballot(a == v);
    list = lane == n ? v : list;
    ++n;
  }
  return n;
}

// 16 MB rows, whose K the four waves share.  Columns are those of the tile's adapters one after the
// other, rank each; a workgroup takes CB blocks of 16, and again every chunks-th.  U steps of 32 of K on
// their way at once; those of x before the adapters are known.
template <int DT, int MB, int CB>
__global__ __launch_bounds__(256) void k_lowrank_down(LowrankArgs g) {
  typedef typename Half<DT>::V8 V8;
  constexpr int U = MB * CB <= 2 ? 8 : 4, KS = 4;
  __shared__ v4f s_part[KS - 1][MB][CB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % g.splits;
  const int rest = blockIdx.x / g.splits;
  const int chunk = rest % g.chunks;
  const int64_t r0 = (int64_t)(rest / g.chunks) * (16 * MB);
  const int rl = lane & 15, kq = lane >> 4;
  int mine[MB];
  const uint16_t* px[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int64_t row = r0 + 16 * m + rl;
    mine[m] = adapter_of(g, row);
    px[m] = g.x + min(row, g.rows - 1) * g.ldx + 8 * kq;
  }
  const int tile_row = adapter_of(g, lane < 16 * MB ? r0 + lane : g.rows);
  const int steps = g.k / 32;
  const int parts = g.splits * KS, part = split * KS + wave;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
  V8 fx[U][MB], next[U][MB];
  auto load_x = [&](int s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < s1) {
#pragma unroll
        for (int m = 0; m < MB; ++m) next[u][m] = *reinterpret_cast<const V8*>(px[m] + 32 * (int64_t)(s + u));
      }
  };
  load_x(s0);
  int list;
  const int nd = distinct(tile_row, list);
  const int cols = nd * g.rank;
  for (int c0 = chunk * CB * 16; c0 < cols; c0 += g.chunks * CB * 16) {  // the same for all waves
    const uint16_t* pw[CB];
#pragma unroll
    for (int b = 0; b < CB; ++b) {
      const int c = min(c0 + 16 * b + rl, cols - 1);
      const int d = c / g.rank;
      const int64_t a = __shfl(list, d, 64);
      pw[b] = g.down + (a * g.rank + (c - d * g.rank)) * g.k + 8 * kq;
    }
    if (c0 != chunk * CB * 16) load_x(s0);
    v4f acc[MB][CB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int b = 0; b < CB; ++b) acc[m][b] = v4f{};
    for (int s = s0; s < s1; s += U) {
      V8 fw[U][CB];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < MB; ++m) fx[u][m] = next[u][m];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s + u < s1) {
#pragma unroll
          for (int b = 0; b < CB; ++b) fw[u][b] = *reinterpret_cast<const V8*>(pw[b] + 32 * (int64_t)(s + u));
        }
      if (s + U < s1) load_x(s + U);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s + u < s1) {
#pragma unroll
          for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int b = 0; b < CB; ++b) acc[m][b] = mfma32<DT>(fw[u][b], fx[u][m], acc[m][b]);
        }
    }
    if (wave) {
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int b = 0; b < CB; ++b) s_part[wave - 1][m][b][lane] = acc[m][b];
    }
    __syncthreads();
    // Lane (rl, kq) has four columns of row rl in each block, all of one adapter (rank % 8 == 0).
    if (!wave) {
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const int c = c0 + 16 * b + 4 * kq;
        const int d = min(c, cols - 1) / g.rank;
        const int a = __shfl(list, d, 64);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
#pragma unroll
          for (int w = 0; w < KS - 1; ++w) acc[m][b] += s_part[w][m][b][lane];
          if (c < cols && a == mine[m])
            *reinterpret_cast<v4f*>(g.t + ((int64_t)split * g.rows + r0 + 16 * m + rl) * g.rank + (c - d * g.rank)) = acc[m][b];
        }
      }
    }
    __syncthreads();
  }
}

// Eight elements of a row, cnt of them inside it, and what they are with v added.
template <int DT>
struct Row8 {
  typename std::conditional<DT == DT_F32, v4f, u4v>::type q[DT == DT_F32 ? 2 : 1];

  __device__ __forceinline__ void load(const void* base, int64_t at, int cnt) {
    if constexpr (DT == DT_F32) {
      const float* b = reinterpret_cast<const float*>(base) + at;
      if (cnt == 8) {
        q[0] = reinterpret_cast<const v4f_el*>(b)[0];
        q[1] = reinterpret_cast<const v4f_el*>(b)[1];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i >> 2][i & 3] = i < cnt ? b[i] : 0.0f;
      }
    } else {
      const uint16_t* b = reinterpret_cast<const uint16_t*>(base) + at;
      q[0] = cnt == 8 ? load8<false, false>(b, 8) : load8<true, false>(b, cnt);
    }
  }
  __device__ __forceinline__ void add(const float* v) {
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i >> 2][i & 3] = q[i >> 2][i & 3] + v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float b0, b1;
        decode2<DT>(q[0][i], b0, b1);
        q[0][i] = cvt_pair<DT>(b0 + v[2 * i], b1 + v[2 * i + 1]);
      }
    }
  }
  __device__ __forceinline__ void store(void* out, int64_t at, int cnt) const {
    if constexpr (DT == DT_F32) {
      float* o = reinterpret_cast<float*>(out) + at;
      if (cnt == 8) {
        reinterpret_cast<v4f_el*>(o)[0] = q[0];
        reinterpret_cast<v4f_el*>(o)[1] = q[1];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < cnt) o[i] = q[i >> 2][i & 3];
      }
    } else {
      uint16_t* o = reinterpret_cast<uint16_t*>(out) + at;
      if (cnt == 8) store8<false, false>(o, q[0], 8);
      else store8<true, false>(o, q[0], cnt);
    }
  }
};

// The larger of an fp16 row's largest |t| and |t|, of which only numbers count.
__device__ __forceinline__ float top_of(float top, float t) { return fabsf(t) < bits_f(0x7F800000u) ? fmaxf(top, fabsf(t)) : top; }
// What brings an fp16 row whose largest |t| is `top` to [2^13, 2^14), and back (bfloat16 has float32's range).
template <int DT>
__device__ __forceinline__ void fit_of(float top, float& fit, float& back) {
  fit = back = 1.0f;
  if constexpr (DT == DT_F16) {
    // (2^126 is the largest scale whose inverse is normal too)
    const int by = min(13 - ((int)(f_bits(top) >> 23) - 127), 126);
    fit = bits_f((unsigned)(127 + by) << 23);
    back = bits_f((unsigned)(127 - by) << 23);
  }
}
// t moved a unit of its last place towards zero (an infinity to the largest number), 0 as it is.
__device__ __forceinline__ unsigned inward(float t) { return f_bits(t) - (t != 0.0f ? 1u : 0u); }
// Two values of t cut off to their upper pieces; t becomes what is left, which is not zero and of t's sign.
template <int DT>
__device__ __forceinline__ unsigned upper(float& t0, float& t1) {
  if constexpr (DT == DT_BF16) {
    const unsigned u0 = inward(t0), u1 = inward(t1);
    t0 -= bits_f(u0 & 0xFFFF0000u);
    t1 -= bits_f(u1 & 0xFFFF0000u);
    return u0 >> 16 | (u1 & 0xFFFF0000u);
  } else {
    // (at least 3 2^-26 is left of all but the smallest, which rounds to 2^-24, the least of fp16)
    const float i0 = bits_f(inward(t0)) - copysignf(0x1.8p-25f, t0), i1 = bits_f(inward(t1)) - copysignf(0x1.8p-25f, t1);
    const unsigned u = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_pkrtz(i0, i1));
    float h0, h1;
    decode2<DT>(u, h0, h1);
    t0 -= h0;
    t1 -= h1;
    return u;
  }
}
// Pieces of t: two; three where a float32 output of bfloat16 operands would show the third (24 bits are t).
template <int DT, int OUT_DT>
constexpr int PIECES = DT == DT_BF16 && OUT_DT == DT_F32 ? 3 : 2;
template <int DT, int N>
__device__ __forceinline__ void pieces(float t0, float t1, unsigned (&p)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; ++i) p[i] = upper<DT>(t0, t1);
  p[N - 1] = cvt_pair<DT>(t0, t1);
}
// A step of 32 of the rank from row q of up: eight elements a lane.
template <typename V8>
__device__ __forceinline__ V8 up_step(const uint16_t* q, int s, int kq, int rank) {
  return 32 * s + 8 * kq < rank ? *reinterpret_cast<const V8*>(q + 32 * s) : V8{};
}
// Row i of the two blocks of 16 rows of up for 32 columns: column 8 (i / 4) + 4 b + i % 4, so that a
// lane's sums are eight consecutive outputs of its row.
__device__ __forceinline__ int up_col(int rl, int b) { return 8 * (rl >> 2) + 4 * b + (rl & 3); }

// Few rows: a wave of its own for 16 rows by 32 columns, t straight into the product's layout.  RS: steps
// of 32 of the rank.  Four steps of up are on their way at once, of as many adapters.
template <int DT, int OUT_DT, int RS>
__global__ __launch_bounds__(64) void k_lowrank_up_few(LowrankArgs g) {
  typedef typename Half<DT>::V8 V8;
  constexpr int DU = 4 / RS, P = PIECES<DT, OUT_DT>;
  const int lane = threadIdx.x, rl = lane & 15, kq = lane >> 4;
  const int64_t row = (int64_t)(blockIdx.x / g.col_tiles) * 16 + rl;
  const int n0 = (int)(blockIdx.x % g.col_tiles) * 32, n = n0 + 8 * kq;
  const bool here = row < g.rows && n < g.n;
  const int mine = adapter_of(g, row);
  v4f t[RS][2];
  const float* pt = g.t + min(row, g.rows - 1) * g.rank + 8 * kq;
#pragma unroll
  for (int s = 0; s < RS; ++s) t[s][0] = t[s][1] = v4f{};
#pragma unroll 4
  for (int q = 0; q < g.splits; ++q) {
#pragma unroll
    for (int s = 0; s < RS; ++s)
      if (32 * s + 8 * kq < g.rank) {
        const v4f* e = reinterpret_cast<const v4f*>(pt + (int64_t)q * g.rows * g.rank + 32 * s);
        t[s][0] += e[0];
        t[s][1] += e[1];
      }
  }
  Row8<OUT_DT> io;
  if (here) io.load(g.base, row * g.ldb + n, min(8, g.n - n));
  int list;
  const int nd = distinct(mine, list);
  const float sc = mine >= 0 && g.scale ? g.scale[mine] : 1.0f;
  float top = 0.0f;
#pragma unroll
  for (int s = 0; s < RS; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[s][i >> 2][i & 3] = t[s][i >> 2][i & 3] * sc;
      if constexpr (DT == DT_F16) top = top_of(top, t[s][i >> 2][i & 3]);
    }
  if constexpr (DT == DT_F16) {
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
  }
  float fit, back;
  fit_of<DT>(top, fit, back);
  V8 part[P][RS];
#pragma unroll
  for (int s = 0; s < RS; ++s) {
    u4v q[P];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unsigned u[P];
      pieces<DT>(t[s][i >> 1][2 * (i & 1)] * fit, t[s][i >> 1][2 * (i & 1) + 1] * fit, u);
#pragma unroll
      for (int p = 0; p < P; ++p) q[p][i] = u[p];
    }
#pragma unroll
    for (int p = 0; p < P; ++p) part[p][s] = __builtin_bit_cast(V8, q[p]);
  }
  for (int d0 = 0; d0 < nd; d0 += DU) {
    V8 fu[DU][RS][2];
#pragma unroll
    for (int u = 0; u < DU; ++u) {
      const int64_t a = __builtin_amdgcn_readlane(list, min(d0 + u, nd - 1));
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint16_t* q = g.up + (a * g.n + min(n0 + up_col(rl, b), g.n - 1)) * g.rank + 8 * kq;
#pragma unroll
        for (int s = 0; s < RS; ++s) fu[u][s][b] = up_step<V8>(q, s, kq, g.rank);
      }
    }
#pragma unroll
    for (int u = 0; u < DU; ++u) {
      if (d0 + u >= nd) break;
      v4f acc[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        acc[b] = v4f{};
#pragma unroll
        for (int s = 0; s < RS; ++s) {
#pragma unroll
          for (int p = P - 1; p >= 0; --p) acc[b] = mfma32<DT>(fu[u][s][b], part[p][s], acc[b]);
        }
      }
      // Each row takes the sums of its own adapter, once.
      if (mine == __builtin_amdgcn_readlane(list, d0 + u)) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = acc[i >> 2][i & 3] * back;
        io.add(v);
      }
    }
  }
  if (here) io.store(g.out, row * g.ldo + n, min(8, g.n - n));
}

// Many rows: 16 MB rows, of which each of the four waves takes 64 columns; t's pieces shared through LDS.
// The sums of 16 rows change places through LDS, so that a load of base and a store of out cover whole
// 128-byte lines of eight rows (from the product's own layout they cover 64 bytes of sixteen rows).
constexpr int UP_WAVES = 4, UP_COLS = 64, UP_PITCH = UP_COLS + 4;

template <int DT, int OUT_DT, int MB, int RS>
__global__ __launch_bounds__(64 * UP_WAVES) void k_lowrank_up(LowrankArgs g) {
  typedef typename Half<DT>::V8 V8;
  constexpr int TP = 32 * RS + 8;  // pitch of t's pieces: eight lanes' rows start in different banks
  constexpr int P = PIECES<DT, OUT_DT>;
  __shared__ __attribute__((aligned(16))) uint16_t s_t[P][16 * MB][TP];
  __shared__ __attribute__((aligned(16))) float s_sum[UP_WAVES][16][UP_PITCH];
  __shared__ float s_back[16 * MB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rl = lane & 15, kq = lane >> 4;
  const int64_t r0 = (int64_t)(blockIdx.x / g.col_tiles) * (16 * MB);
  const int n0 = ((int)(blockIdx.x % g.col_tiles) * UP_WAVES + wave) * UP_COLS;
  const int tile_row = adapter_of(g, lane < 16 * MB ? r0 + lane : g.rows);

  // t of the tile: sixteen lanes a row, one row of each 16, asked for before base.
  constexpr int CH = RS > 2 ? 2 : 1;
  const int tr = threadIdx.x >> 4;
  v4f t[MB][CH];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int j = 0; j < CH; ++j) t[mb][j] = v4f{};
#pragma unroll 4
  for (int q = 0; q < g.splits; ++q) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const float* p = g.t + (q * g.rows + min(r0 + 16 * mb + tr, g.rows - 1)) * g.rank;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = 4 * (rl + 16 * j);
        if (c < g.rank) t[mb][j] += *reinterpret_cast<const v4f*>(p + c);
      }
    }
  }
  int list;
  const int nd = distinct(tile_row, list);
  V8 fu[2][2][RS];
  auto load_up = [&](int d) {
    const int64_t a = __builtin_amdgcn_readlane(list, d);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint16_t* q = g.up + (a * g.n + min(n0 + 32 * p + up_col(rl, b), g.n - 1)) * g.rank + 8 * kq;
#pragma unroll
        for (int s = 0; s < RS; ++s) fu[p][b][s] = up_step<V8>(q, s, kq, g.rank);
      }
  };
  if (nd) load_up(0);
  // Piece j of the lane's outputs: row 8 j + lane / 8 of the tile, columns from `col`.
  const int col = n0 + 8 * (lane & 7);
  Row8<OUT_DT> io[2 * MB];
#pragma unroll
  for (int j = 0; j < 2 * MB; ++j) {
    const int64_t row = r0 + 8 * j + (lane >> 3);
    if (row < g.rows && col < g.n) io[j].load(g.base, row * g.ldb + col, min(8, g.n - col));
  }
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int a = adapter_of(g, r0 + 16 * mb + tr);
    const float sc = a >= 0 && g.scale ? g.scale[a] : 1.0f;
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t[mb][j][i] = t[mb][j][i] * sc;
        if constexpr (DT == DT_F16) top = top_of(top, t[mb][j][i]);
      }
    if constexpr (DT == DT_F16) {
      top = fmaxf(top, dpp_f<0xB1>(top));
      top = fmaxf(top, dpp_f<0x4E>(top));
      top = fmaxf(top, dpp_f<0x141>(top));
      top = fmaxf(top, dpp_f<0x140>(top));
    }
    float fit, back;
    fit_of<DT>(top, fit, back);
    if (rl == 0) s_back[16 * mb + tr] = back;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = 4 * (rl + 16 * j);
      if (c < 32 * RS) {
        u2v q[P];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          unsigned u[P];
          pieces<DT>(t[mb][j][2 * i] * fit, t[mb][j][2 * i + 1] * fit, u);
#pragma unroll
          for (int p = 0; p < P; ++p) q[p][i] = u[p];
        }
#pragma unroll
        for (int p = 0; p < P; ++p) *reinterpret_cast<u2v*>(&s_t[p][16 * mb + tr][c]) = q[p];
      }
    }
  }
  __syncthreads();
  if (n0 >= g.n) return;
  float (*sums)[UP_PITCH] = s_sum[wave];
  for (int d = 0; d < nd; ++d) {
    const int a = __builtin_amdgcn_readlane(list, d);
    if (d) load_up(d);
    const uint64_t rows_of_a = __ballot(tile_row == a);
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      if (!((rows_of_a >> (16 * mb)) & 0xFFFF)) continue;
      v4f acc[2][2];
#pragma unroll
      for (int p = 0; p < 2; ++p) acc[p][0] = acc[p][1] = v4f{};
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        V8 part[P];
#pragma unroll
        for (int p = 0; p < P; ++p) part[p] = *reinterpret_cast<const V8*>(&s_t[p][16 * mb + rl][32 * s + 8 * kq]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int p = P - 1; p >= 0; --p) acc[c][b] = mfma32<DT>(fu[c][b][s], part[p], acc[c][b]);
          }
      }
      const float back = s_back[16 * mb + rl];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int b = 0; b < 2; ++b) *reinterpret_cast<v4f*>(&sums[rl][32 * p + 8 * kq + 4 * b]) = acc[p][b] * back;
      __builtin_amdgcn_wave_barrier();
      // Each row takes the sums of its own adapter, once.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * h + (lane >> 3);
        if ((rows_of_a >> (16 * mb + r)) & 1) {
          const v4f* q = reinterpret_cast<const v4f*>(&sums[r][8 * (lane & 7)]);
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = q[i >> 2][i & 3];
          io[2 * mb + h].add(v);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
#pragma unroll
  for (int j = 0; j < 2 * MB; ++j) {
    const int64_t row = r0 + 8 * j + (lane >> 3);
    if (row < g.rows && col < g.n) io[j].store(g.out, row * g.ldo + col, min(8, g.n - col));
  }
}

}  // namespace vqk

namespace vq_internal {

using namespace vqk;

namespace {
constexpr int64_t DOWN_GROUPS = 512;  // two workgroups a compute unit
constexpr int64_t MAX_PARTS = 8, PART_K = 512;
// Rows of t in the scratch, over all parts of K.  A buffer made for a larger call (more rows, adapters, rank or
// K) has to do for a smaller one, whose plan may have more parts, so this is no plan's own product but
// what none exceeds: parts are at most MAX_PARTS and K / PART_K, and a plan with more than one has at most
// 2 DOWN_GROUPS workgroups, each of at most 32 rows.
int64_t lowrank_t_rows(int64_t rows, int64_t k) {
  return std::max(rows, std::min(std::min(MAX_PARTS, std::max<int64_t>(1, k / PART_K)) * rows, 2 * DOWN_GROUPS * 32));
}
// How the first product is cut: tiles of 16 or 32 rows by blocks of 16 columns, workgroups of their own for
// further columns, and for parts of K, while rows alone do not fill the compute units.
struct LowrankPlan {
  int mb, cb, chunks, splits;
  int64_t tiles;
};
LowrankPlan lowrank_plan(int64_t rows, int adapters, int rank, int64_t k) {
  LowrankPlan p;
  rows = std::max<int64_t>(1, rows);
  // Tiles of 32 rows read the adapters half as often: where they still fill the compute units (17776 rows,
  // 1920, rank 32, 33 -> 31 us, rank 128 90 -> 73; but 4000 rows of rank 32 14 -> 18), and for large ranks
  // (1000 rows of rank 128 20 -> 15).
  p.mb = rows >= 8192 || (rank > 64 && rows > 16) ? 2 : 1;
  p.tiles = (rows + 16 * p.mb - 1) / (16 * p.mb);
  p.cb = rank <= 32 ? 2 : 4;
  const int64_t cols = (int64_t)std::min<int64_t>(std::min<int64_t>(16 * p.mb, rows), adapters) * rank;
  p.chunks = (int)std::min<int64_t>((cols + 16 * p.cb - 1) / (16 * p.cb), std::max<int64_t>(1, DOWN_GROUPS / p.tiles));
  // Parts of 512 of K up to two workgroups a compute unit, of 2048 up to four (5159 rows, 7424, 323 tiles: three
  // parts 44 -> 32 us; 13439 rows, 3520, 420 tiles: two parts 25 -> 27).  The second product adds up to eight.
  const int64_t groups = p.tiles * p.chunks;
  p.splits = (int)std::max<int64_t>({1, std::min<int64_t>({MAX_PARTS, DOWN_GROUPS / groups, k / PART_K}),
                                     std::min<int64_t>({MAX_PARTS, 2 * DOWN_GROUPS / groups, k / 2048})});
  return p;
}
}  // namespace

int64_t lowrank_workspace_elems(int64_t rows, int64_t rank, int64_t k) {
  return lowrank_t_rows(std::max<int64_t>(1, rows), k) * rank;
}

int64_t lowrank_groups(int64_t rows, int64_t adapters, int64_t rank, int64_t k, int64_t n) {
  const LowrankPlan p = lowrank_plan(rows, (int)adapters, (int)rank, k);
  return std::max(p.tiles * p.chunks * p.splits, (rows + 31) / 32 * ((n + 255) / 256));
}

template <int DT>
static void launch_down(const LowrankArgs& a, const LowrankPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.tiles * p.chunks * p.splits));
  auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(256), 0, st, a); };
  if (p.mb == 1) {
    if (p.cb == 2) go(k_lowrank_down<DT, 1, 2>);
    else go(k_lowrank_down<DT, 1, 4>);
  } else {
    if (p.cb == 2) go(k_lowrank_down<DT, 2, 2>);
    else go(k_lowrank_down<DT, 2, 4>);
  }
}

template <int DT, int OUT_DT, int RS>
static void launch_up_rs(LowrankArgs a, hipStream_t st) {
  // Waves of their own, shared tiles of 16 rows, of 32 (us, 1920 -> 5760, rank 32: 64 rows 4.0, 4.8, 7.6; 200 rows
  // 7.6, 5.2, 7.0; 1000 rows 13.2, 8.4, 8.9; 17776 rows -, 97, 87; fewer rows a tile read up more often).
  // Tiles of 64 rows are no faster (17776 rows 92, rank 128 even).
  const int mb = a.rows <= 64 ? 0 : a.rows < 1024 ? 1 : 2;
  const int rows = mb == 2 ? 32 : 16, cols = mb ? UP_WAVES * UP_COLS : 32;
  a.col_tiles = (a.n + cols - 1) / cols;
  const dim3 grid((unsigned)((a.rows + rows - 1) / rows * a.col_tiles));
  if (mb == 2) hipLaunchKernelGGL((k_lowrank_up<DT, OUT_DT, 2, RS>), grid, dim3(64 * UP_WAVES), 0, st, a);
  else if (mb == 1) hipLaunchKernelGGL((k_lowrank_up<DT, OUT_DT, 1, RS>), grid, dim3(64 * UP_WAVES), 0, st, a);
  else hipLaunchKernelGGL((k_lowrank_up_few<DT, OUT_DT, RS>), grid, dim3(64), 0, st, a);
}
template <int DT, int OUT_DT>
static void launch_up(const LowrankArgs& a, hipStream_t st) {
  if (a.rank <= 32) launch_up_rs<DT, OUT_DT, 1>(a, st);
  else if (a.rank <= 64) launch_up_rs<DT, OUT_DT, 2>(a, st);
  else launch_up_rs<DT, OUT_DT, 4>(a, st);
}

template <int DT>
static void launch_lowrank_dt(const LowrankArgs& a, const LowrankPlan& p, int out_dt, hipStream_t st) {
  launch_down<DT>(a, p, st);
  if (out_dt == DT_F32) launch_up<DT, DT_F32>(a, st);
  else launch_up<DT, DT>(a, st);
}

hipError_t launch_lowrank(const LowrankParams& p, hipStream_t st) {
  LowrankArgs a{};
  a.x = reinterpret_cast<const uint16_t*>(p.x);
  a.down = reinterpret_cast<const uint16_t*>(p.down);
  a.up = reinterpret_cast<const uint16_t*>(p.up);
  a.index = p.index;
  a.scale = p.scale;
  a.base = p.base;
  a.out = p.out;
  a.t = p.t;
  a.ldx = p.ldx;
  a.ldb = p.ldb;
  a.ldo = p.ldo;
  a.rows = p.rows;
  a.adapters = (int)p.adapters;
  a.rank = (int)p.rank;
  a.k = (int)p.k;
  a.n = (int)p.n;
  const LowrankPlan plan = lowrank_plan(p.rows, a.adapters, a.rank, p.k);
  a.splits = plan.splits;
  a.chunks = plan.chunks;
  if (p.dtype == DT_BF16) launch_lowrank_dt<DT_BF16>(a, plan, p.out_dt, st);
  else launch_lowrank_dt<DT_F16>(a, plan, p.out_dt, st);
  return hipGetLastError();
}

}  // namespace vq_internal
