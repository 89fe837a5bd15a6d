// Matrix products of several experts in one launch for gfx950: the rows of A, sorted by
// expert, meet the weights of their own expert.  Two kinds share the tiling: int8 codes
// times packed 8-bit or 4-bit weight codes with the dequantizing epilogue of the integer
// GEMM (the same arithmetic, so a row's output equals that GEMM's bit for bit), and
// 16-bit rows times 16-bit weights with float32 accumulation.
//
// The rows' distribution is known on the device only: offsets[e] .. offsets[e + 1] are
// expert e's rows.  A launch is sized by the number of rows and experts alone, and a
// workgroup finds its tiles from the offsets: k_experts_few from a prefix sum of the experts'
// tile counts, 64 experts per wave step, k_experts_pp from a table of it in LDS.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "dev_common.h"
#include "gemm_common.h"
#include "vq_internal.h"

namespace vqk {

// Wide stores at any element's address (the hardware takes unaligned ones): an odd number of
// outputs leaves every other row unaligned.  Stored element by element, 8190 rows of 16-bit
// elements over 8 experts, 2048 -> 5759, took 370 us instead of 281.  Only those at a multiple of two
// bytes that is none of four are slow, so the large tiles avoid them: 260 -> 239 us (5758: 236).
typedef u4v u4v_any __attribute__((aligned(2)));
typedef u2v u2v_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

// Operand kinds.
enum : int { X_I8 = 0, X_I4 = 1, X_F16 = 2, X_BF16 = 3 };

struct XArgs {
  const uint8_t* a;       // rows of codes or 16-bit elements
  const float* sa;        // per row of a
  const uint8_t* b;       // weights of all experts
  const float* sb;        // per expert and output
  const int32_t* off;     // [experts + 1]
  const int32_t* rows;    // row of a for each output row, or nullptr
  void* y;
  int experts, m_a, t, n, k;
  int64_t lda, ldb;       // bytes from one row to the next
  int64_t b_expert;       // bytes from one expert's weights to the next
  int64_t b_piece;        // bytes from one 64-byte K piece to the next (64: row-major)
  int64_t ldy;
  int max_items;          // tiles of 256 x 256 that ascending offsets can have at most
};

// The tile-th row tile of BM rows over all experts: its expert, first row and the
// expert's last row + 1.  False past the last tile.  Every lane returns the same values.
// Offsets are clamped to [0, t], so any values keep the rows inside the buffers.
struct RowTile {
  int e, r0, r1;
};
__device__ __forceinline__ bool find_tile(const XArgs& g, int bm, int tile, RowTile& out) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < g.experts; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < g.experts) {
      lo = min(max(g.off[e], 0), g.t);
      hi = min(max(g.off[e + 1], 0), g.t);
    }
    const int nt = hi > lo ? (hi - lo + bm - 1) / bm : 0;
    int inc = nt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(inc, o, 64);
      if (lane >= o) inc += u;
    }
    const int total = __shfl(inc, 63, 64);
    if (tile < base + total) {
      const uint64_t hit = __ballot(base + inc > tile);
      const int l = __builtin_ctzll(hit);
      out.e = __builtin_amdgcn_readfirstlane(e0 + l);
      const int first = base + __shfl(inc, l, 64) - __shfl(nt, l, 64);
      out.r0 = __builtin_amdgcn_readfirstlane(__shfl(lo, l, 64) + (tile - first) * bm);
      out.r1 = __builtin_amdgcn_readfirstlane(__shfl(hi, l, 64));
      return true;
    }
    base += total;
  }
  return false;
}

// ---------------------------------------------------------------------------------------
// Few rows per expert (decoding): a product is bound by the weights' bytes, and each is
// needed by one tile only.  A workgroup owns 16 rows of outputs and 32 columns for each of
// its 4 / KS column groups; KS waves share a group's K, with both operands straight from
// memory into registers (no LDS and no barriers in the K loop), and their sums are joined
// through LDS.  A 16-row fragment load covers whole 64-byte pieces of the weights, 1 KB in
// all; with the weights in K pieces that is one contiguous block.  Two pieces a batch:
// four take registers, and with them waves (16 rows over 16 experts, 1920 -> 5760, 4-bit:
// 19.9 against 14.6 us).  Measured: 24 rows over 8 experts, 4096 -> 1920, 16-bit, 24.8 us = 4.9 TB/s
// of weights; the 4-bit case above 12.8 us = 4.4 TB/s.
constexpr int FEW_STEPS = 2;   // 64-byte pieces of weights in a batch; two batches in flight
constexpr int FEW_M = 16, FEW_N = 32;

template <int KIND, int OUT_DT, int KS>
__global__ __launch_bounds__(256) void k_experts_few(XArgs g, int tiles_n) {
  constexpr bool INT = KIND == X_I8 || KIND == X_I4;
  constexpr int AP = KIND == X_I4 ? 2 : 1;  // fragments of A for a piece of weights
  typedef typename std::conditional<KIND == X_BF16, __bf16, _Float16>::type in_t;
  typedef in_t in8 __attribute__((ext_vector_type(8)));
  typedef typename std::conditional<INT, v4i, v4f>::type acc_t;
  typedef typename std::conditional<INT, int, float>::type el_t;
  __shared__ acc_t s_part[4][2][64];
  RowTile tl;
  const int tm = blockIdx.x / tiles_n;
  if (!find_tile(g, FEW_M, tm, tl)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rl = lane & 15, kq = lane >> 4;
  const int kw = wave % KS;
  const int n0 = (((int)blockIdx.x - tm * tiles_n) * (4 / KS) + wave / KS) * FEW_N;
  const int row = tl.r0 + rl;
  const bool row_ok = row < tl.r1;
  int ar = row_ok ? row : tl.r0;
  if (g.rows) ar = g.rows[ar];
  const uint8_t* pb[2];
#pragma unroll
  for (int b = 0; b < 2; ++b)
    pb[b] = g.b + tl.e * g.b_expert + (int64_t)min(n0 + 16 * b + rl, g.n - 1) * g.ldb + 16 * kq;
  // Pieces of a weight row: 64 bytes each, the last one of a 4-bit row possibly half.
  const int pieces = KIND == X_I8 ? g.k / 64 : KIND == X_I4 ? (g.k + 127) / 128 : g.k / 32;
  const int p0 = pieces * kw / KS, p1 = pieces * (kw + 1) / KS;
  acc_t acc[2] = {acc_t{}, acc_t{}};
  v4i fa[2][FEW_STEPS][AP], fb[2][FEW_STEPS][2];
  auto load_b = [&](int set, int p) {
#pragma unroll
    for (int u = 0; u < FEW_STEPS; ++u) {
      const int q = min(p + u, p1 - 1);  // past the end: a valid piece, not used
      // the half piece's second half lies past a 4-bit row: its first half again, against zeros
      const int back = KIND == X_I4 && 128 * q + 32 * kq >= g.k ? 32 : 0;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        fb[set][u][b] = *reinterpret_cast<const v4i*>(pb[b] + (int64_t)q * g.b_piece - back);
      }
    }
  };
  if (p0 < p1) load_b(0, p0);
  const bool a_ok = (unsigned)ar < (unsigned)g.m_a;  // an index outside a gives a row of zeros
  ar = a_ok ? ar : 0;
  const uint8_t* pa = g.a + ar * g.lda + 16 * AP * kq;
  auto load_a = [&](int set, int p) {
#pragma unroll
    for (int u = 0; u < FEW_STEPS; ++u) {
      const int q = min(p + u, p1 - 1);
#pragma unroll
      for (int h = 0; h < AP; ++h) {
        if (KIND == X_I4 && 128 * q + 32 * kq >= g.k) fa[set][u][h] = v4i{0, 0, 0, 0};
        else fa[set][u][h] = *reinterpret_cast<const v4i*>(pa + 64 * AP * q + 16 * h);
      }
    }
  };
  auto mma = [&](int set, int p) {
#pragma unroll
    for (int u = 0; u < FEW_STEPS; ++u) {
      if (p + u >= p1) break;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const v4i w = fb[set][u][b];
        if constexpr (KIND == X_I4) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(unpack_int4x16(h ? u2v{(unsigned)w.z, (unsigned)w.w} : u2v{(unsigned)w.x, (unsigned)w.y}), fa[set][u][h], acc[b], 0, 0, 0);
        } else if constexpr (KIND == X_I8) {
          acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, fa[set][u][0], acc[b], 0, 0, 0);
        } else if constexpr (KIND == X_F16) {
          acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(in8, w), __builtin_bit_cast(in8, fa[set][u][0]), acc[b], 0, 0, 0);
        } else {
          acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(in8, w), __builtin_bit_cast(in8, fa[set][u][0]), acc[b], 0, 0, 0);
        }
      }
    }
  };
  if (p0 < p1) {
    load_a(0, p0);
    for (int p = p0; p < p1; p += 2 * FEW_STEPS) {
      if (p + FEW_STEPS < p1) {
        load_b(1, p + FEW_STEPS);
        load_a(1, p + FEW_STEPS);
      }
      mma(0, p);
      if (p + 2 * FEW_STEPS < p1) {
        load_b(0, p + 2 * FEW_STEPS);
        load_a(0, p + 2 * FEW_STEPS);
      }
      mma(1, p + FEW_STEPS);
    }
  }
  // Lane l of a 16 x 16 block holds row l mod 16 and columns 4 (l div 16) + 0..3.  The
  // first two waves of a K split finish a block each.
  if constexpr (KS > 1) {
#pragma unroll
    for (int b = 0; b < 2; ++b) s_part[wave][b][lane] = acc[b];
    __syncthreads();
  }
  const float sa = INT ? g.sa[ar] : 1.0f;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if (KS > 1 && kw != b) continue;
    const int nq = n0 + 16 * b + 4 * kq;
    if (!row_ok || nq >= g.n) continue;
    const int cnt = min(4, g.n - nq);
    acc_t v = acc[b];
    if constexpr (KS > 1) {
      v = s_part[wave - kw][b][lane];
#pragma unroll
      for (int w = 1; w < KS; ++w) v += s_part[wave - kw + w][b][lane];
    }
    float out[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      el_t x = v[r];
      if constexpr (INT) {
        if constexpr (KIND == X_I4) x >>= 4;
        out[r] = (float)x * (sa * g.sb[(int64_t)tl.e * g.n + min(nq + r, g.n - 1)]);
      } else {
        out[r] = x;
      }
      if (!a_ok) out[r] = 0.0f;
    }
    const int64_t o = (int64_t)row * g.ldy + nq;
    if constexpr (OUT_DT == DT_F32) {
      float* dst = reinterpret_cast<float*>(g.y) + o;
      if (cnt == 4) {
        *reinterpret_cast<v4f_any*>(dst) = v4f{out[0], out[1], out[2], out[3]};
      } else {
        for (int r = 0; r < cnt; ++r) dst[r] = out[r];
      }
    } else {
      const unsigned q0 = cvt_pair<OUT_DT>(out[0], out[1]), q1 = cvt_pair<OUT_DT>(out[2], out[3]);
      uint16_t* dst = reinterpret_cast<uint16_t*>(g.y) + o;
      if (cnt == 4) {
        *reinterpret_cast<u2v_any*>(dst) = u2v{q0, q1};
      } else {
        for (int r = 0; r < cnt; ++r) dst[r] = (uint16_t)((r < 2 ? q0 : q1) >> (16 * (r & 1)));
      }
    }
  }
}

template <int KIND, int KS>
static hipError_t launch_few_split(const XArgs& a, int out_dt, hipStream_t st) {
  const int64_t tiles = a.t / FEW_M + (a.experts < a.t ? a.experts : a.t);
  const int tiles_n = (a.n + FEW_N * (4 / KS) - 1) / (FEW_N * (4 / KS));
  const dim3 grid((unsigned)(tiles * tiles_n));
  switch (out_dt) {
    case DT_F16: hipLaunchKernelGGL((k_experts_few<KIND, DT_F16, KS>), grid, dim3(256), 0, st, a, tiles_n); break;
    case DT_BF16: hipLaunchKernelGGL((k_experts_few<KIND, DT_BF16, KS>), grid, dim3(256), 0, st, a, tiles_n); break;
    default: hipLaunchKernelGGL((k_experts_few<KIND, DT_F32, KS>), grid, dim3(256), 0, st, a, tiles_n); break;
  }
  return hipGetLastError();
}

template <int KIND>
static hipError_t launch_few_kind(const XArgs& a, int out_dt, hipStream_t st) {
  // Four waves on K, two where a row has so few pieces that a quarter is three or less
  // (16 rows over 16 experts, 1920 -> 5760, 4-bit: 12.9 us against 14.6; 24 rows over 8,
  // 4096 -> 1920, 16-bit: 32.8 against 24.7).
  const int pieces = KIND == X_I8 ? a.k / 64 : KIND == X_I4 ? a.k / 128 : a.k / 32;
  return pieces < 16 ? launch_few_split<KIND, 2>(a, out_dt, st) : launch_few_split<KIND, 4>(a, out_dt, st);
}

// ---------------------------------------------------------------------------------------
// Many rows per expert: 256 x 256 output tiles on the ping-pong schedule of the single
// layers (k_qgemm_pp, k_gemm_dense): 8 waves, the two of a SIMD alternating between a
// memory phase (the fragment reads of a 64-byte K stage and its share of the direct loads
// two stages ahead) and a compute phase (that stage's MFMAs from registers).
//
// Ragged shares: an expert's last tile has any number of rows, so a wave's four 32-row
// blocks are spread over the tile (block 2 mb + wm) and a tile of NM * 64 rows at most runs
// a K loop of NM blocks per wave: its matrix time follows its rows, in steps of 64, waves
// load no rows that are not there, and only the weights' traffic is that of a whole tile.
//
// Tiles: the experts' tile counts are summed into a table in LDS once per workgroup (about
// 3 us with the first loads); a wave finds a tile's expert with two ballots over it.  The rows'
// indices of a tile are requested a whole tile ahead of their use.  Whole tiles come first,
// the experts' last ones after them; the tiles of a last round that would leave half of the
// grid idle are cut in two or four: by rows, or where they have 128 at most by columns,
// since the time of a short tile is that of its weights (64 rows, 8192 -> 16384: 84 us whole,
// 54 in four).
//
// Measured: 17776 rows over 8 experts, 1920 -> 5760, 8-bit, 234 us = 1.68 POP/s; 6001 over 4,
// 12288 -> 1920, 4-bit, 162 us = 1.74; 8190 over 8, 2048 -> 5759, 16-bit, 243 us = 0.80 PFLOP/s (237
// for 5760; 191 for one expert: 1.01, whose 736 tiles are 2.9 rounds of 256, where the eight experts'
// 830 to 850 are 3.3 and the last round's pieces each walk all of K).  With 8-bit and 4-bit codes the
// matrix units' power sets the rate of whole tiles: dealing the last tiles out evenly by their
// measured cost changed nothing.  4124 rows over 32
// experts, 2048 -> 2048, 8-bit: 54 us, where the weights alone take 27: a first round of 256 tiles
// at 4 TB/s and a second one that is bound by the latency of its stages.
namespace xp {
constexpr int BM = 256, BN = 256, NT = 512;
constexpr int WTN = 64, MBLK = 4, NBLK = 2;
constexpr int ROW = 64;                  // bytes of an A row per stage: 64 codes or 32 elements
constexpr int NST = 4, D = 2;
constexpr int A_BYTES = BM * ROW;
constexpr int LA = A_BYTES / (NT * 16);  // direct loads per wave and stage (2)
}  // namespace xp

// Row scales of an index outside a and of 16-bit rows.  No row's own scale is -0.
__device__ const float x_none = -0.0f, x_one = 1.0f;

template <int KIND, int OUT_DT>
__global__ __launch_bounds__(xp::NT) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_experts_pp(XArgs g) {
  using namespace xp;
  constexpr bool INT = KIND == X_I8 || KIND == X_I4;
  constexpr bool HALF_OUT = OUT_DT != DT_F32;
  constexpr int B_ROW = KIND == X_I4 ? 32 : 64;
  constexpr int STAGE = A_BYTES + BN * B_ROW;
  constexpr int LB = BN * B_ROW / (NT * 16);
  constexpr int L = LA + LB;
  typedef typename std::conditional<KIND == X_BF16, __bf16, _Float16>::type in_t;
  typedef in_t in8 __attribute__((ext_vector_type(8)));
  typedef typename std::conditional<INT, v16i, v16f>::type acc_t;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NST * STAGE];
  __shared__ float s_sa[2][BM];
  __shared__ float s_sb[2][BN];
  extern __shared__ int s_tab[];  // [experts] each: sums of whole tiles and of tails up to an expert, its rows
  const int E = g.experts;
  int* s_whole = s_tab;
  int* s_tail = s_tab + E;
  int* s_lo = s_tab + 2 * E;
  int* s_hi = s_tab + 3 * E;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2;  // waves w and w + 4 share a SIMD
  const int wm = wave & 1, wn = wave >> 1;
  const int nk = INT ? g.k / 64 : g.k / 32;

  if (wave == 0) {
    int whole = 0, tails = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      int lo = 0, hi = 0;
      if (e < E) {
        lo = min(max(g.off[e], 0), g.t);
        hi = min(max(g.off[e + 1], 0), g.t);
      }
      const int len = hi > lo ? hi - lo : 0;
      int inc = len / BM;
      const uint64_t has_tail = __ballot(len % BM != 0);
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(inc, o, 64);
        if (lane >= o) inc += u;
      }
      if (e < E) {
        s_whole[e] = whole + inc;
        s_tail[e] = tails + __builtin_popcountll(has_tail & (~0ull >> (63 - lane)));
        s_lo[e] = lo;
        s_hi[e] = hi;
      }
      whole += __shfl(inc, 63, 64);
      tails += __builtin_popcountll(has_tail);
    }
  }
  __syncthreads();
  const int whole_m = __builtin_amdgcn_readfirstlane(s_whole[E - 1]);
  const int tiles_m = whole_m + __builtin_amdgcn_readfirstlane(s_tail[E - 1]);
  const int tiles_n = (g.n + BN - 1) / BN;
  if ((int64_t)tiles_m * tiles_n > g.max_items) return;  // offsets that do not ascend
  const int tiles = tiles_m * tiles_n;
  const int rest = tiles % (int)gridDim.x;
  const int split = 4 * rest <= (int)gridDim.x ? 4 : 2 * rest <= (int)gridDim.x ? 2 : 1;
  const int whole_items = tiles - rest;
  // Whole tiles come first, so in the last round the workgroups with the highest numbers
  // have had the short ones: they take its pieces.
  const int G = (int)gridDim.x;
  const int last = G - 1 - (int)blockIdx.x;  // this workgroup's piece of the last round, if there are so many
  int t = blockIdx.x;
  auto next_item = [&](int w) {  // the item after w (-1: none)
    if (w >= 0 && w < whole_items && w + G < whole_items) return w + G;
    return w < whole_items && last < rest * split ? whole_items + last : -1;
  };
  if (t >= whole_items) t = next_item(whole_items - 1);
  if (t < 0) return;

  struct Tile {
    int e, r0, rows, n0, cols;
  };
  const int chunk = (E + 63) / 64;
  auto locate = [&](int w) {
    const int j = max(w - whole_items, 0);  // past the whole rounds: piece j % split of a tile
    const int part = j % split;
    int tm, tn;
    tile_of(w < whole_items ? w : whole_items + j / split, tiles_m, tiles_n, tm, tn);
    const bool tail = tm >= whole_m;
    const int* cnt = tail ? s_tail : s_whole;
    const int want = tail ? tm - whole_m : tm;
    const uint64_t h0 = __ballot(cnt[min((lane + 1) * chunk, E) - 1] > want);
    const int c0 = __builtin_ctzll(h0) * chunk;
    const uint64_t h1 = __ballot(cnt[min(c0 + lane, E - 1)] > want);
    Tile x;
    x.e = c0 + __builtin_ctzll(h1);
    const int lo = __builtin_amdgcn_readfirstlane(s_lo[x.e]), hi = __builtin_amdgcn_readfirstlane(s_hi[x.e]);
    const int before = !tail && x.e ? __builtin_amdgcn_readfirstlane(s_whole[x.e - 1]) : 0;
    // A piece is a part of the tile's columns where the rows are few (the time is then that
    // of the weights), else of its rows.
    const int r0 = tail ? hi - (hi - lo) % BM : lo + (want - before) * BM;
    const int rows = min(BM, hi - r0);
    const bool pieces = w >= whole_items, by_cols = pieces && rows <= 128;
    const int step = pieces && !by_cols ? BM / split : BM;
    x.cols = by_cols ? BN / split : BN;
    x.r0 = r0 + (pieces && !by_cols ? part * step : 0);
    x.n0 = tn * BN + (by_cols ? part * x.cols : 0);
    x.rows = x.n0 < g.n ? min(step, r0 + rows - x.r0) : 0;  // <= 0: an empty piece
    return x;
  };

  int ra[LA], ca[LA], rb[LB], cb[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) dma_lane<ROW>(wave * LA + i, lane, ra[i], ca[i]);
#pragma unroll
  for (int i = 0; i < LB; ++i) dma_lane<B_ROW>(wave * LB + i, lane, rb[i], cb[i]);
  const int rs = 64 * (wave & 3) + lane;  // the row or column whose scale this lane loads
  int ia[LA], is = 0;                     // rows of a: of this lane's loads, of its scale
  auto request_rows = [&](const Tile& x) {
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r = x.r0 + min(ra[i], x.rows - 1);
      ia[i] = g.rows ? g.rows[r] : r;
    }
    const int r = x.r0 + min(rs, x.rows - 1);
    is = g.rows ? g.rows[r] : r;
  };
  const uint8_t* ga[LA];
  const uint8_t* gb[LB];
  int64_t boff = 0;
  auto set_tile = [&](const Tile& x) {
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r = (unsigned)ia[i] < (unsigned)g.m_a ? ia[i] : 0;
      ga[i] = g.a + r * g.lda + ca[i];
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) gb[i] = g.b + x.e * g.b_expert + (int64_t)min(x.n0 + rb[i], g.n - 1) * g.ldb + cb[i];
    boff = 0;
  };
  // Row scales (x_none for an index outside a; 1 for 16-bit rows) and column scales, by direct
  // loads ahead of the tile's first stage.
  auto load_scales = [&](const Tile& x, int buf) {
    if (wave < 4) {
      const bool ok = (unsigned)is < (unsigned)g.m_a;
      const float* src = !ok ? &x_none : INT ? g.sa + is : &x_one;
      dma4(src, &s_sa[buf][64 * wave]);
    } else {
      const float* src = INT ? g.sb + (int64_t)x.e * g.n + min(x.n0 + rs, g.n - 1) : &x_one;
      dma4(src, &s_sb[buf][64 * (wave - 4)]);
    }
  };
  // A wave loads 32 rows of A; the waves past a tile's last 64-row block load none.
  // Likewise 32 rows of B, and none past a piece's columns.
  auto issue = [&](int s, bool with_a, bool with_b) {  // called for s = 0, 1, 2, ... of a tile in order
    uint8_t* base = lds + (s % NST) * STAGE;
    if (with_a) {
#pragma unroll
      for (int i = 0; i < LA; ++i) dma16(ga[i] + s * ROW, base + (wave * LA + i) * 1024);
    }
    if (with_b) {
#pragma unroll
      for (int i = 0; i < LB; ++i) dma16(gb[i] + boff, base + A_BYTES + (wave * LB + i) * 1024);
    }
    if constexpr (KIND == X_I4) boff += (s & 1) ? g.b_piece - 32 : 32;
    else boff += g.b_piece;
  };

  const int rl = lane & 31, kc = lane >> 5;
  int fa[2], fb[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    fa[h] = (wm * 32 + rl) * ROW + 16 * ((2 * h + kc) ^ swz64(rl));
    if constexpr (KIND == X_I4) fb[h] = A_BYTES + (wn * WTN + rl) * B_ROW + 16 * (h ^ swz32(rl)) + 8 * kc;
    else fb[h] = A_BYTES + (wn * WTN + rl) * B_ROW + 16 * ((2 * h + kc) ^ swz64(rl));
  }
  acc_t acc[MBLK][NBLK];
  typedef typename std::conditional<KIND == X_I4, u2v, v4i>::type b_t;
  v4i fA[2][MBLK];
  b_t fB[2][NBLK];
  // Rows that start at an odd element store their pieces of eight columns one column to the left
  // (but the wave's first piece; the last column by itself), so that they start at four bytes.
  const bool odd = HALF_OUT && ((g.ldy & 1) || (reinterpret_cast<uintptr_t>(g.y) & 2));
  bool pend = false;  // the previous tile's 16 stores follow this tile's first loads

  // The K loop of a tile whose rows need NM blocks per wave.
  auto k_loop = [&](auto nm_c, int cols) {
    constexpr int NM = decltype(nm_c)::value;
    const bool with_a = NM == MBLK || wave < 2 * NM;
    const bool with_b = NM > 2 || 32 * wave < cols, active = NM > 2 || WTN * wn < cols;
    auto wait_next = [&](bool stores) {  // every load but the last stage's done
      if (stores) wait_vmcnt<(D - 1) * L + 16>();  // whole tiles only: every wave then has L loads a stage
      else if (with_a && with_b) wait_vmcnt<(D - 1) * L>();
      else if (with_b) wait_vmcnt<(D - 1) * LB>();
      else wait_vmcnt<(D - 1) * LA>();  // (a wave without loads waits for nothing)
    };
    auto wait_groups = [&](int later) {
      if (later < 1) wait_vmcnt<0>();
      else wait_next(false);
    };
    auto read_stage = [&](int slot) {
      const uint8_t* base = lds + slot * STAGE;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int nb = 0; nb < NBLK; ++nb) fB[h][nb] = *reinterpret_cast<const b_t*>(base + fb[h] + nb * 32 * B_ROW);
#pragma unroll
        for (int mb = 0; mb < NM; ++mb) fA[h][mb] = *reinterpret_cast<const v4i*>(base + fa[h] + mb * 64 * ROW);
      }
    };
    auto compute = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nb = 0; nb < NBLK; ++nb) {
          v4i b;
          if constexpr (KIND == X_I4) b = unpack_int4x16(fB[h][nb]);
          else b = fB[h][nb];
#pragma unroll
          for (int mb = 0; mb < NM; ++mb) {
            if constexpr (INT)
              acc[mb][nb] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b, fA[h][mb], acc[mb][nb], 0, 0, 0);
            else if constexpr (KIND == X_F16)
              acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(in8, b), __builtin_bit_cast(in8, fA[h][mb]), acc[mb][nb], 0, 0, 0);
            else
              acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(in8, b), __builtin_bit_cast(in8, fA[h][mb]), acc[mb][nb], 0, 0, 0);
          }
        }
    };
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
      for (int j = 0; j < NBLK; ++j) acc[i][j] = acc_t{};
    if (pend && NM == MBLK && nk > D) wait_next(true);
    else wait_groups(min(D, nk) - 1);
    sched_barrier_all();
    if (grp == 1) sched_barrier_all();
    int p = 0;
    for (; p + D < nk; ++p) {
      if (active) read_stage(p % NST);
      issue(p + D, with_a, with_b);
      const bool early = pend && NM == MBLK && p < D - 1;  // stage p + 1 was loaded before the stores
      if (grp == 1) wait_next(early);
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      sched_barrier_all();
      if (active) compute();
      if (grp == 0) wait_next(early);
      sched_barrier_all();
    }
    for (; p < nk; ++p) {
      if (active) read_stage(p % NST);
      const int later = nk - p - 2;
      if (grp == 1) wait_groups(later);
      __builtin_amdgcn_s_waitcnt(0xC07F);
      sched_barrier_all();
      if (active) compute();
      if (grp == 0) wait_groups(later);
      sched_barrier_all();
    }
    if (grp == 0) sched_barrier_all();
  };

  Tile cur = locate(t), nxt = cur;
  if (cur.rows <= 0) return;  // only a workgroup's last item can be empty
  request_rows(cur);
  set_tile(cur);
  load_scales(cur, 0);
  t = next_item(t);
  bool more = t >= 0;
  if (more) {
    nxt = locate(t);
    more = nxt.rows > 0;
    if (more) request_rows(nxt);
  }
#pragma unroll
  for (int s = 0; s < D; ++s)
    if (s < nk) issue(s, wave < 2 * ((cur.rows + 63) / 64), 32 * wave < cur.cols);
  int buf = 0;
  typedef typename std::conditional<OUT_DT == DT_BF16, __bf16, _Float16>::type h_t;
  for (;;) {
    const int nm = (cur.rows + 63) / 64;
    if (nm == 4) k_loop(std::integral_constant<int, 4>{}, cur.cols);
    else if (nm == 3) k_loop(std::integral_constant<int, 3>{}, cur.cols);
    else if (nm == 2) k_loop(std::integral_constant<int, 2>{}, cur.cols);
    else k_loop(std::integral_constant<int, 1>{}, cur.cols);

    const bool has_next = more;
    const Tile c = cur;
    if (has_next) {
      cur = nxt;
      set_tile(cur);
      load_scales(cur, buf ^ 1);
      t = next_item(t);
      more = t >= 0;
      if (more) {
        nxt = locate(t);
        more = nxt.rows > 0;
        if (more) request_rows(nxt);
      }
#pragma unroll
      for (int s = 0; s < D; ++s)
        if (s < nk) issue(s, wave < 2 * ((cur.rows + 63) / 64), 32 * wave < cur.cols);
    }
    const bool full = c.rows == BM && c.n0 + BN <= g.n;  // (of all columns: pieces by columns have few rows)
    pend = HALF_OUT && has_next && full;
    v4f sb_r[NBLK][4];
    if constexpr (INT) {
#pragma unroll
      for (int nb = 0; nb < NBLK; ++nb)
#pragma unroll
        for (int q = 0; q < 4; ++q) sb_r[nb][q] = *reinterpret_cast<const v4f*>(&s_sb[buf][wn * WTN + 4 * kc + nb * 32 + 8 * q]);
    }
#pragma unroll
    for (int mb = 0; mb < MBLK; ++mb) {
      if (mb >= nm || WTN * wn >= c.cols) break;
      const int ml = 64 * mb + 32 * wm + rl;
      const int m = c.r0 + ml;
      const float sa0 = s_sa[buf][ml];
      // Zeros for an index outside a, also where a column's scale or a row of a is not finite.
      const bool none = f_bits(sa0) == 0x80000000u, some_none = __any(none);
      const bool shift = odd && (((int64_t)(reinterpret_cast<uintptr_t>(g.y) >> 1) + m * g.ldy) & 1);
      unsigned before = 0;  // the eight columns before this lane's: the last two
#pragma unroll
      for (int nb = 0; nb < NBLK; ++nb) {
        unsigned pk[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = c.n0 + wn * WTN + 4 * kc + nb * 32 + 8 * q;
          float out[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (INT) {
              int a0 = acc[mb][nb][4 * q + r];
              if constexpr (KIND == X_I4) a0 >>= 4;
              const float t0 = sa0 * sb_r[nb][q][r];
              out[r] = (float)a0 * t0;
            } else {
              out[r] = acc[mb][nb][4 * q + r];
            }
          }
          if constexpr (HALF_OUT) {
            pk[2 * q] = cvt_pair<OUT_DT>(out[0], out[1]);
            pk[2 * q + 1] = cvt_pair<OUT_DT>(out[2], out[3]);
          } else {
            if (some_none) {
#pragma unroll
              for (int r = 0; r < 4; ++r) out[r] = none ? 0.0f : out[r];
            }
            float* dst = reinterpret_cast<float*>(g.y) + (int64_t)m * g.ldy + n;
            if (ml < c.rows && n + 4 <= g.n) {
              *reinterpret_cast<v4f_any*>(dst) = v4f{out[0], out[1], out[2], out[3]};
            } else if (ml < c.rows) {
              for (int r = 0; r < 4 && n + r < g.n; ++r) dst[r] = out[r];
            }
          }
        }
        if constexpr (HALF_OUT) {
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const auto s0 = __builtin_amdgcn_permlane32_swap(pk[4 * pr], pk[4 * pr + 2], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(pk[4 * pr + 1], pk[4 * pr + 3], false, false);
            u4v w = {s0[0], s1[0], s0[1], s1[1]};
            if (some_none) w = none ? u4v{0u, 0u, 0u, 0u} : w;
            const int no = c.n0 + wn * WTN + nb * 32 + 16 * pr + 8 * kc;
            h_t* dst = reinterpret_cast<h_t*>(g.y) + (int64_t)m * g.ldy + no;
            u4v wide = w;
            h_t* to = dst;
            if (odd) {
              const auto last = __builtin_amdgcn_permlane32_swap(w.w, w.w, false, false);
              const unsigned left = kc ? last[0] : before;
              before = last[1];
              if (shift && nb + pr + kc > 0) {
                wide = u4v{__builtin_amdgcn_alignbit(w.x, left, 16), __builtin_amdgcn_alignbit(w.y, w.x, 16),
                           __builtin_amdgcn_alignbit(w.z, w.y, 16), __builtin_amdgcn_alignbit(w.w, w.z, 16)};
                --to;
              }
              // The last column, where no further piece of this wave is stored whole.
              if (shift && ((nb == NBLK - 1 && pr + kc == 2) || no + 16 > g.n) && ml < c.rows && no + 8 <= g.n)
                dst[7] = __builtin_bit_cast(h_t, (unsigned short)(w.w >> 16));
            }
            if (full) {
              *reinterpret_cast<u4v_any*>(to) = wide;
            } else if (ml < c.rows && no < g.n) {
              if (no + 8 <= g.n) {
                *reinterpret_cast<u4v_any*>(to) = wide;
              } else {
                for (int e = 0; e < 8 && no + e < g.n; ++e) {
                  const unsigned d = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
                  dst[e] = __builtin_bit_cast(h_t, (unsigned short)(d >> (16 * (e & 1))));
                }
              }
            }
          }
        }
      }
    }
    if (!has_next) break;
    buf ^= 1;
  }
}

template <int KIND>
static hipError_t launch_pp_kind(XArgs a, int out_dt, hipStream_t st) {
  const int64_t tiles = (a.t / xp::BM + (a.experts < a.t ? a.experts : a.t)) * (int64_t)((a.n + xp::BN - 1) / xp::BN);
  a.max_items = (int)tiles;  // at most (2^18 + 2^10) * 2^12 (the entry point's limits)
  const int pb = vq_internal::persistent_blocks();
  const dim3 grid((unsigned)std::min<int64_t>(4 * tiles, pb));  // a tile may be cut in four
  const size_t shm = (size_t)a.experts * 16;  // at most 16 KB beside the 132 KB of the ring and scales
  switch (out_dt) {
    case DT_F16: hipLaunchKernelGGL((k_experts_pp<KIND, DT_F16>), grid, dim3(xp::NT), shm, st, a); break;
    case DT_BF16: hipLaunchKernelGGL((k_experts_pp<KIND, DT_BF16>), grid, dim3(xp::NT), shm, st, a); break;
    default: hipLaunchKernelGGL((k_experts_pp<KIND, DT_F32>), grid, dim3(xp::NT), shm, st, a); break;
  }
  return hipGetLastError();
}

template <int KIND>
static hipError_t launch_kind(const XArgs& a, int out_dt, hipStream_t st) {
  // The few-row kernel reads the weights again for every 16 rows; the other one needs
  // about as many 256-column tiles as compute units to reach the memory's rate.  Measured
  // over 32 experts, 2048 -> 2048 (256 such tiles), us: 8-bit weights, 4 / 8 / 16 rows each,
  // 28.4 / 29.8 / 37.8 against 29.1 / 29.5 / 30.3; 4-bit 16.9 / 19.0 / 25.1 against 20.1 /
  // 20.8 / 20.7; 16-bit 50.6 / 55.0 / 73.0 against 67.9 / 67.8 / 68.8.  With fewer tiles the
  // rows from which the other one wins grow a little more slowly than their number falls:
  // 64 tiles (8 experts, 4096 -> 2048), 16 / 32 rows each, 19.1 / 29.2 against 21.4 / 21.5,
  // 14.3 / 21.0 against 25.0 / 25.1, 39.0 / 58.6 against 54.1 / 54.2; 16 tiles (2 experts), 64
  // rows each, 18.1 against 23.2, 13.2 against 27.6, 32.6 against 41.0.  The rule is a power law through
  // three numbers of tiles and takes the slower kernel at two of these points: 16 tiles, 8-bit, 64 rows
  // each (it turns at 48), and 64 tiles, 4-bit, 32 rows each (at 28).
  const int64_t used = std::min<int64_t>(a.experts, a.t);
  const int64_t cus = vq_internal::persistent_blocks();
  const int64_t tiles = std::min<int64_t>(used * ((a.n + xp::BN - 1) / xp::BN), cus);
  const int64_t few_tiles = (a.t / FEW_M + used) * ((a.n + FEW_N - 1) / FEW_N);
  const double few_rows = (KIND == X_I8 ? 6.0 : 10.0) * std::pow((double)cus / (double)tiles, 0.75);
  if ((double)a.t > few_rows * (double)a.experts || few_tiles > (1 << 23))
    return launch_pp_kind<KIND>(a, out_dt, st);
  return launch_few_kind<KIND>(a, out_dt, st);
}

}  // namespace vqk

namespace vq_internal {

using namespace vqk;

hipError_t launch_experts(const ExpertsParams& p, hipStream_t st) {
  XArgs a{};
  a.a = reinterpret_cast<const uint8_t*>(p.a);
  a.sa = p.sa;
  a.b = reinterpret_cast<const uint8_t*>(p.b);
  a.sb = p.sb;
  a.off = p.offsets;
  a.rows = p.rows;
  a.y = p.y;
  a.experts = (int)p.experts;
  a.m_a = (int)p.m_a;
  a.t = (int)p.t;
  a.n = (int)p.n;
  a.k = (int)p.k;
  a.lda = p.lda;
  a.ldb = p.ldb;
  a.b_expert = p.b_expert;
  a.b_piece = p.b_piece;
  a.ldy = p.ldy;
  switch (p.kind) {
    case X_I8: return launch_kind<X_I8>(a, p.out_dt, st);
    case X_I4: return launch_kind<X_I4>(a, p.out_dt, st);
    case X_F16: return launch_kind<X_F16>(a, p.out_dt, st);
    default: return launch_kind<X_BF16>(a, p.out_dt, st);
  }
}

}  // namespace vq_internal
