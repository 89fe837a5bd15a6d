// Low-rank adapters of many requests beside a projection that they share, for gfx950:
//
//   out[i] = RNE(base[i] + scale[a] * (x[i] . down[a]^T) . up[a]^T),   a = index[i]
//
// over rows whose requests use different adapters, or none (index -1: out[i] = base[i]).  The inner
// dimension, the rank, is small, so the products are bound by the bytes of x, base and out
// (and, for few rows, of the adapters); both run on the matrix cores.
//   k_lowrank_down  t = x . down^T: 16 rows a tile, against the columns of the adapters that
//                   its rows use, each once; K in parts where rows are few.  Sums in float32.
//   k_lowrank_up    out = base + t . up^T: a tile goes through the adapters of its rows one after the
//                   other, and each row takes the one that is its own.  Sums of different adapters do
//                   not meet, so an infinity or NaN in one adapter stays out of the other requests' rows.
// t, scaled, enters the second product as the sum of two 16-bit values (hi = RNE16(t), lo = RNE16(t - hi)):
// rounded once it would cost the output up to 2^-9 of the adapter's part in bfloat16, in two
// pieces 2^-17 (fp16 2^-22), for a second matrix instruction in a kernel that waits for memory.  An
// fp16 row is scaled by the power of two that brings its largest |t| to [2^13, 2^14), since t is not bound to
// fp16's range; the products are scaled back, both exactly (a lo below 2^-24 is lost).
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
  float* t;  // [splits, rows, rank]
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

// Columns are those of the tile's adapters one after the other, rank each, CB blocks of 16 a
// workgroup.  KS waves share a tile's K (1: each of the four has a tile of its own).
template <int DT, int CB, int KS>
__global__ __launch_bounds__(256) void k_lowrank_down(LowrankArgs g) {
  typedef typename Half<DT>::V8 V8;
  __shared__ v4f s_part[KS > 1 ? KS : 1][CB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % g.splits;
  const int rest = blockIdx.x / g.splits;
  const int chunk = rest % g.chunks;
  const int64_t tile = KS > 1 ? rest / g.chunks : (int64_t)(rest / g.chunks) * 4 + wave;
  const int kw = KS > 1 ? wave : 0;
  const int rl = lane & 15, kq = lane >> 4;
  const int64_t row = tile * 16 + rl;
  const int mine = adapter_of(g, row);
  int list;
  const int nd = distinct(mine, list);
  const int cols = nd * g.rank;
  const int c0 = chunk * CB * 16;
  if (c0 >= cols) return;  // the same for a tile's waves
  const uint16_t* px = g.x + min(row, g.rows - 1) * g.ldx + 8 * kq;
  const uint16_t* pw[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) {
    const int c = min(c0 + 16 * b + rl, cols - 1);
    const int d = c / g.rank;
    const int64_t a = __shfl(list, d, 64);
    pw[b] = g.down + (a * g.rank + (c - d * g.rank)) * g.k + 8 * kq;
  }
  const int steps = g.k / 32;
  const int parts = g.splits * KS, part = split * KS + kw;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
  v4f acc[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) acc[b] = v4f{};
  constexpr int U = CB <= 2 ? 8 : 4;
  for (int s = s0; s < s1; s += U) {
    V8 fx[U], fw[U][CB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t e = 32 * (int64_t)min(s + u, s1 - 1);
      fx[u] = *reinterpret_cast<const V8*>(px + e);
#pragma unroll
      for (int b = 0; b < CB; ++b) fw[u][b] = *reinterpret_cast<const V8*>(pw[b] + e);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < s1) {
#pragma unroll
        for (int b = 0; b < CB; ++b) acc[b] = mfma32<DT>(fw[u][b], fx[u], acc[b]);
      }
  }
  if constexpr (KS > 1) {
#pragma unroll
    for (int b = 0; b < CB; ++b) s_part[kw][b][lane] = acc[b];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int b = 0; b < CB; ++b)
#pragma unroll
      for (int w = 1; w < KS; ++w) acc[b] += s_part[w][b][lane];
  }
  // Lane (rl, kq) has four columns of row rl in each block, all of one adapter (rank % 8 == 0).
#pragma unroll
  for (int b = 0; b < CB; ++b) {
    const int c = c0 + 16 * b + 4 * kq;
    const int d = min(c, cols - 1) / g.rank;
    const int a = __shfl(list, d, 64);
    if (c < cols && a == mine)
      *reinterpret_cast<v4f*>(g.t + ((int64_t)split * g.rows + row) * g.rank + (c - d * g.rank)) = acc[b];
  }
}

#ifndef UP_MB
#define UP_MB 2
#define UP_NP 2
#define UP_MANY 1024
#endif
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

// Waves side by side, each 16 MB rows by 32 NP columns.  RS: steps of 32 of the rank.  DU: adapters whose
// rows of up are on their way at once.  LINES: the sums change places through LDS, so that a load of
// base and a store of out cover whole 128-byte lines of eight rows (from the product's own
// layout they cover 64 bytes of sixteen rows).
template <int DT, int OUT_DT, int MB, int NP, int RS, int DU, bool LINES>
__global__ __launch_bounds__(256) void k_lowrank_up(LowrankArgs g) {
  typedef typename Half<DT>::V8 V8;
  static_assert(!LINES || NP == 2, "eight lanes of eight columns a row");
  constexpr int COLS = 32 * NP, PITCH = COLS + 4;
  extern __shared__ __attribute__((aligned(16))) float s_sum[];  // LINES: [waves][16 MB][PITCH]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rl = lane & 15, kq = lane >> 4;
  const int64_t r0 = (int64_t)(blockIdx.x / g.col_tiles) * (16 * MB);
  const int n0 = ((int)(blockIdx.x % g.col_tiles) * (int)(blockDim.x >> 6) + wave) * COLS;
  if (n0 >= g.n) return;

  // Piece j of the lane's outputs: its row in the tile and its column.
  auto row_of = [&](int j) { return LINES ? 8 * j + (lane >> 3) : 16 * (j / NP) + rl; };
  auto col_of = [&](int j) { return n0 + (LINES ? 8 * (lane & 7) : 32 * (j % NP) + 8 * kq); };
  int mine[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) mine[mb] = adapter_of(g, r0 + 16 * mb + rl);
  const int tile_row = adapter_of(g, lane < 16 * MB ? r0 + lane : g.rows);
  // t: asked for first, and used last of what is asked for here.
  V8 hi[MB][RS], lo[MB][RS];
  float back[MB];
  v4f t[MB][RS][2];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const float* p = g.t + min(r0 + 16 * mb + rl, g.rows - 1) * g.rank + 8 * kq;
#pragma unroll
    for (int s = 0; s < RS; ++s) {
      t[mb][s][0] = t[mb][s][1] = v4f{};
      if (32 * s + 8 * kq < g.rank)
        for (int q = 0; q < g.splits; ++q) {
          const v4f* e = reinterpret_cast<const v4f*>(p + (int64_t)q * g.rows * g.rank + 32 * s);
          t[mb][s][0] += e[0];
          t[mb][s][1] += e[1];
        }
    }
  }
  Row8<OUT_DT> io[MB * NP];
#pragma unroll
  for (int j = 0; j < MB * NP; ++j)
    if (r0 + row_of(j) < g.rows && col_of(j) < g.n)
      io[j].load(g.base, (r0 + row_of(j)) * g.ldb + col_of(j), min(8, g.n - col_of(j)));
  int list;
  const int nd = distinct(tile_row, list);

  // t, scaled, in two pieces.
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const float sc = mine[mb] >= 0 && g.scale ? g.scale[mine[mb]] : 1.0f;
    float top = 0.0f;
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = t[mb][s][i >> 2][i & 3] * sc;
        t[mb][s][i >> 2][i & 3] = v;
        top = fmaxf(top, fabsf(v));
      }
    float fit = 1.0f;
    back[mb] = 1.0f;
    if constexpr (DT == DT_F16) {
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      // 2^(13 - exponent of the largest); without a finite, normal one nothing is scaled
      const int e = (int)(f_bits(top) >> 23) - 127;
      const int by = top < bits_f(0x7F800000u) && e > -100 && e < 100 ? 13 - e : 0;
      fit = bits_f((unsigned)(127 + by) << 23);
      back[mb] = bits_f((unsigned)(127 - by) << 23);
    }
#pragma unroll
    for (int s = 0; s < RS; ++s) {
      u4v h, l;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float t0 = t[mb][s][i >> 1][2 * (i & 1)] * fit, t1 = t[mb][s][i >> 1][2 * (i & 1) + 1] * fit;
        h[i] = cvt_pair<DT>(t0, t1);
        float h0, h1;
        decode2<DT>(h[i], h0, h1);
        // an infinite hi has no rest
        const float d0 = fabsf(h0) < bits_f(0x7F800000u) ? t0 - h0 : 0.0f;
        const float d1 = fabsf(h1) < bits_f(0x7F800000u) ? t1 - h1 : 0.0f;
        l[i] = cvt_pair<DT>(d0, d1);
      }
      hi[mb][s] = __builtin_bit_cast(V8, h);
      lo[mb][s] = __builtin_bit_cast(V8, l);
    }
  }

  float* sums = s_sum + wave * (16 * MB * PITCH);
  for (int d0 = 0; d0 < nd; d0 += DU) {
    V8 fu[DU][RS][NP][2];
#pragma unroll
    for (int u = 0; u < DU; ++u) {
      const int64_t a = __builtin_amdgcn_readlane(list, min(d0 + u, nd - 1));
      // Row i of block b is column 8 (i / 4) + 4 b + i % 4, so that a lane's sums are eight
      // consecutive outputs of its row.
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int n = min(n0 + 32 * p + 8 * (rl >> 2) + 4 * b + (rl & 3), g.n - 1);
          const uint16_t* q = g.up + (a * g.n + n) * g.rank + 8 * kq;
#pragma unroll
          for (int s = 0; s < RS; ++s) {
            fu[u][s][p][b] = V8{};
            if (32 * s + 8 * kq < g.rank) fu[u][s][p][b] = *reinterpret_cast<const V8*>(q + 32 * s);
          }
        }
    }
#pragma unroll
    for (int u = 0; u < DU; ++u) {
      if (d0 + u >= nd) break;
      const int a = __builtin_amdgcn_readlane(list, d0 + u);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        v4f acc[NP][2];
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            acc[p][b] = v4f{};
#pragma unroll
            for (int s = 0; s < RS; ++s) {
              acc[p][b] = mfma32<DT>(fu[u][s][p][b], lo[mb][s], acc[p][b]);
              acc[p][b] = mfma32<DT>(fu[u][s][p][b], hi[mb][s], acc[p][b]);
            }
          }
        // Each row takes the sums of its own adapter, once.
        if (mine[mb] == a) {
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            if constexpr (LINES) {
#pragma unroll
              for (int b = 0; b < 2; ++b)
                *reinterpret_cast<v4f*>(sums + (16 * mb + rl) * PITCH + 32 * p + 8 * kq + 4 * b) = acc[p][b] * back[mb];
            } else {
              float v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = acc[p][i >> 2][i & 3] * back[mb];
              io[mb * NP + p].add(v);
            }
          }
        }
      }
    }
  }
  if constexpr (LINES) __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < MB * NP; ++j) {
    const int64_t row = r0 + row_of(j);
    if constexpr (LINES) {
      const int own = __shfl(tile_row, row_of(j), 64);
      if (own >= 0) {
        float v[8];
        const v4f* q = reinterpret_cast<const v4f*>(sums + row_of(j) * PITCH + 8 * (lane & 7));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = q[i >> 2][i & 3];
        io[j].add(v);
      }
    }
    if (row < g.rows && col_of(j) < g.n) io[j].store(g.out, row * g.ldo + col_of(j), min(8, g.n - col_of(j)));
  }
}

}  // namespace vqk

namespace vq_internal {

using namespace vqk;

namespace {
// How a call is cut: tiles of 16 rows whose K is shared by four waves (and by `splits` workgroups)
// while rows are few, else a tile a wave.
struct LowrankPlan {
  bool few;
  int cb, chunks, splits;
};
LowrankPlan lowrank_plan(int64_t rows, int adapters, int rank, int64_t k) {
  LowrankPlan p;
  rows = std::max<int64_t>(1, rows);
  const int64_t tiles = (rows + 15) / 16;
  p.few = tiles < 8192;
  const int blocks = (rank + 15) / 16;
  p.cb = blocks <= 2 ? 2 : blocks <= 4 || p.few ? 4 : 8;
  const int64_t cols = (int64_t)std::min<int64_t>(std::min<int64_t>(16, rows), adapters) * rank;
  p.chunks = (int)((cols + 16 * p.cb - 1) / (16 * p.cb));
  p.splits = 1;
  if (p.few) {
    const int64_t most = std::max<int64_t>(1, 512 / (tiles * p.chunks));
    p.splits = (int)std::min<int64_t>(std::min<int64_t>(8, most), std::max<int64_t>(1, k / 512));
  }
  return p;
}
}  // namespace

int64_t lowrank_workspace_elems(int64_t rows, int64_t adapters, int64_t rank, int64_t k) {
  return std::max<int64_t>(1, rows) * rank * lowrank_plan(rows, (int)adapters, (int)rank, k).splits;
}

int64_t lowrank_groups(int64_t rows, int64_t adapters, int64_t rank, int64_t k, int64_t n) {
  const LowrankPlan p = lowrank_plan(rows, (int)adapters, (int)rank, k);
  return std::max((rows + 15) / 16 * p.chunks * p.splits, (rows + 15) / 16 * ((n + 31) / 32));
}

template <int DT>
static void launch_down(const LowrankArgs& a, const LowrankPlan& p, hipStream_t st) {
  const int64_t tiles = (a.rows + 15) / 16;
  const int64_t groups = p.few ? tiles : (tiles + 3) / 4;
  const dim3 grid((unsigned)(groups * p.chunks * p.splits));
  auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(256), 0, st, a); };
  if (p.few) {
    if (p.cb == 2) go(k_lowrank_down<DT, 2, 4>);
    else go(k_lowrank_down<DT, 4, 4>);
  } else {
    if (p.cb == 2) go(k_lowrank_down<DT, 2, 1>);
    else if (p.cb == 4) go(k_lowrank_down<DT, 4, 1>);
    else go(k_lowrank_down<DT, 8, 1>);
  }
}

template <int DT, int OUT_DT, int RS>
static void launch_up_rs(LowrankArgs a, hipStream_t st) {
  const bool many = a.rows >= UP_MANY;
  constexpr int MB = UP_MB, NP = UP_NP, DU = 4 / RS;
  const int mb = many ? MB : 1, waves = many ? 4 : 1, cols = 32 * (many ? NP : 1) * waves;
  a.col_tiles = (a.n + cols - 1) / cols;
  const dim3 grid((unsigned)((a.rows + 16 * mb - 1) / (16 * mb) * a.col_tiles));
  if (many) {
    const size_t lds = (size_t)4 * waves * 16 * MB * (32 * NP + 4);
    hipLaunchKernelGGL((k_lowrank_up<DT, OUT_DT, MB, NP, RS, 1, true>), grid, dim3(64 * waves), lds, st, a);
  } else {
    hipLaunchKernelGGL((k_lowrank_up<DT, OUT_DT, 1, 1, RS, DU, false>), grid, dim3(64), 0, st, a);
  }
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
