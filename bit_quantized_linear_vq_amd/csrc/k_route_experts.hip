// Routing to experts and back for gfx950: from the router's scores to rows sorted by expert (what
// the experts' products take), and from the experts' rows to their tokens again.
//
// Routing.  p = softmax or sigmoid of a row of scores; the choice goes by p + bias (by the scores
// themselves without a bias: the same order, with no rounding), in the groups whose best one or two
// sum highest; ties go to the lower index.  Whole numbers come out, so scores are compared as they are, exact in
// float32, and p (+ bias) in float64: two values may differ by less than float32 holds, and the exponentials
// are some tens of instructions against a launch.
//   k_route_select  a wave (or 16 of its lanes) a row: choices, weights, and the block's count for
//                   each expert
//   k_route_place   offsets, and each choice's place: rows before it in its expert's segment, by
//                   ascending token and choice.  Counts are whole numbers, so the order of their sums does not
//                   matter, and places are the same in every call.
//   k_route_few     both for a few rows: 64 of up to 64 experts, 16 of 256, 4 of more
// Bound by latency and by instructions (17776 rows of 160 scores are 11 MB): a row's exponentials, and for
// each choice a maximum over the row's lanes.  Sixteen lanes a row, since the maximum's steps are then
// register moves that four rows share (a wave a row: 17776 x 160 28 us instead of 14).  The exponentials of a
// softmax's sum are float64 too: by the hardware's float32 2^x they take 1.5 us less there, and put 2^-22 on weights
// that are not renormalised.  By p with more than 160 experts a lane's keys and p no longer fit its 128 registers
// (of a workgroup of 1024): 8 to 164 bytes a lane go through scratch.
//
// Measured: 17776 rows of 160, softmax, six choices, 13.5 + 10.3 us; 4124 of 96 in six groups, sigmoid with
// a bias, four choices, 10.6 + 7.9 us; 4096 of 256 in eight, eight choices, 20.7 + 11.6 us; one row of 16 3.7 us.  The placing waits for loads one after the
// other: every block's counts and its choices, then LDS.
#include <algorithm>
#include <type_traits>

#include "dev_common.h"
#include "gemm_common.h"
#include "rows_common.h"
#include "vq_internal.h"

namespace vqk {

struct RouteArgs {
  const void* x;
  const float* bias;  // or nullptr
  int64_t ldx;
  int64_t rows;
  int dtype, experts, top, groups, keep, best, softmax, renorm;
  double scale;
  int32_t* offsets;
  int32_t* row_of;  // [rows * top]
  float* weights;   // [rows, top]
  int32_t* chosen;  // [rows, top]
  int32_t* place;   // [rows, top]
  int32_t* counts;  // [blocks, count_pitch], 16-byte aligned
};


// All lanes of a row (LPR of them) get the same; register moves inside 16 lanes.
template <typename K, int CTRL>
__device__ __forceinline__ K moved(K v) {
  if constexpr (sizeof(K) == 8) return dpp_d<CTRL>(v);
  else return __builtin_bit_cast(K, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
template <int LPR, typename F>
__device__ __forceinline__ void over_row(F&& step) {
  step(std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
  step(std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
  step(std::integral_constant<int, 0x141>{});  // row_half_mirror
  step(std::integral_constant<int, 0x140>{});  // row_mirror
  if constexpr (LPR == 64) {
    step(std::integral_constant<int, -16>{});
    step(std::integral_constant<int, -32>{});
  }
}
template <int CTRL, typename K>
__device__ __forceinline__ K other(K v) {
  if constexpr (CTRL < 0) return __shfl_xor(v, -CTRL, 64);
  else return moved<K, CTRL>(v);
}
template <typename K>
__device__ __forceinline__ K larger(K a, K b) {
  return a > b ? a : b;
}
template <typename K>
__device__ __forceinline__ K smaller(K a, K b) {
  return a > b ? b : a;
}
template <int LPR, typename K>
__device__ __forceinline__ K sum_of(K v) {
  over_row<LPR>([&](auto c) { v += other<decltype(c)::value>(v); });
  return v;
}
template <int LPR, typename K>
__device__ __forceinline__ K max_of(K v) {
  over_row<LPR>([&](auto c) { v = larger(other<decltype(c)::value>(v), v); });
  return v;
}
template <int LPR>
__device__ __forceinline__ int min_of(int v) {
  over_row<LPR>([&](auto c) { v = min(v, other<decltype(c)::value>(v)); });
  return v;
}
// The row's lanes of a ballot, from bit 0.
template <int LPR>
__device__ __forceinline__ uint64_t row_ballot(bool b) {
  const uint64_t m = __ballot(b);
  if constexpr (LPR == 64) return m;
  else return (m >> (threadIdx.x & 63 & ~(LPR - 1))) & ((1ull << LPR) - 1);
}

// e^x in float64: 2^n e^r with n = rne(x / ln 2), |r| <= ln 2 / 2, and e^r by its series to r^13
// (the rest is below 2^-57 of it).  A third of the instructions of the library's function.
__device__ __forceinline__ double exp_d(double x) {
  x = fmin(fmax(x, -800.0), 800.0);  // beyond: 0 and infinity, as the true value rounds
  const double n = __builtin_rint(x * 1.4426950408889634);
  // ln 2 = 190530846196 / 2^38 and a rest: n times the first is exact
  double r = __builtin_fma(n, 190530846196.0 * -0x1p-38, x);
  r = __builtin_fma(n, -1.64659495828970823e-12, r);
  double p = 1.0 / 6227020800.0;
  p = __builtin_fma(p, r, 1.0 / 479001600.0);
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// What the choice goes by.  BY_SCORE: the scores themselves, exact in float32.  BY_P: p (+ bias), in
// float64 for every expert.
enum : int { BY_SCORE = 0, BY_P = 1 };

// A row's choices: lane l of its LPR holds choices l and l + LPR (of experts l + LPR i, in the loop).
// Returned: their experts (-1: none) and weights.  s_row: 8-byte aligned, for groups: experts + groups keys.
template <int LPR, int VPT, int BY, bool SOFT, bool GROUPS>
__device__ __forceinline__ void route_row(const RouteArgs& a, int64_t row, int l, void* s_row, int ch[2], float wt[2]) {
  typedef typename std::conditional<BY == BY_P, double, float>::type K;
  constexpr K NONE = -(K)__builtin_huge_val();
  // What depends on the lane alone stays in the loop over rows: moved out of it, it is held in registers.
  asm volatile("" : "+v"(l));
  float x[VPT];
  auto load = [&](auto dt) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) x[i] = load1<decltype(dt)::value>(a.x, row * a.ldx + min(l + LPR * i, a.experts - 1));
  };
  if (a.dtype == DT_F32) load(std::integral_constant<int, DT_F32>{});
  else if (a.dtype == DT_BF16) load(std::integral_constant<int, DT_BF16>{});
  else load(std::integral_constant<int, DT_F16>{});
  float top = -__builtin_huge_valf();
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    x[i] = l + LPR * i < a.experts ? x[i] : -__builtin_huge_valf();
    bad |= x[i] != x[i] || (SOFT && x[i] == __builtin_huge_valf());
    top = x[i] > top ? x[i] : top;
  }
  double base = 0.0;
  if constexpr (SOFT) {
    top = max_of<LPR>(top);
    base = top > -__builtin_huge_valf() ? (double)top : 0.0;
  }
  // p of every expert where the choice needs it, else their sum where the weights do (of a softmax that
  // is divided by the sum of its chosen they do not).  Without branches, and two exponentials at a time:
  // more of them side by side cost registers, and with them waves.
  double p[BY == BY_P ? VPT : 1];
  double per = 1.0;
  if (SOFT && (BY == BY_P || !a.renorm)) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const double t = exp_d((double)x[i] - base);
      if constexpr (BY == BY_P) p[i] = t;
      sum += t;
      if (i & 1) __builtin_amdgcn_sched_barrier(0);
    }
    sum = sum_of<LPR>(sum);
    per = sum > 0.0 ? 1.0 / sum : 1.0;
  }
  K key[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    key[i] = (K)x[i];
    if constexpr (BY == BY_P) {
      p[i] = SOFT ? p[i] * per : 1.0 / (1.0 + exp_d(-(double)x[i]));
      // (by p without a bias the groups go by p, the choice in them by the scores)
      const double c = a.bias ? p[i] + (double)a.bias[min(l + LPR * i, a.experts - 1)] : (double)x[i];
      key[i] = key[i] == NONE ? NONE : c;
      p[i] = a.bias || key[i] == NONE ? key[i] : p[i];
      bad |= key[i] != key[i];
      if (!SOFT && (i & 1)) __builtin_amdgcn_sched_barrier(0);
    }
  }
  bad = row_ballot<LPR>(bad) != 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) key[i] = bad ? NONE : key[i];
  if constexpr (GROUPS) {
    const int size = a.experts / a.groups;
    const float inv = 1.0f / (float)size;
    // of at most 1024 experts: half a member off a whole number is more than float32's error
    auto group_of = [&](int i) { return (int)(((float)(l + LPR * i) + 0.5f) * inv); };
    // Through LDS, so that a lane goes through members of one group: groups side by side (made up to a
    // power of two), each shared by as many lanes as there are.  A key between the groups that is none
    // keeps their members in different banks.
    K* keys = reinterpret_cast<K*>(s_row);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (l + LPR * i < a.experts) {
        if constexpr (BY == BY_P) keys[l + LPR * i + group_of(i)] = bad ? NONE : p[i];
        else keys[l + LPR * i + group_of(i)] = key[i];
      }
    __builtin_amdgcn_wave_barrier();
    constexpr int SLOTS = 64 / LPR;
    const int lanes = a.groups > LPR / 2 ? LPR : 1 << (32 - __builtin_clz(a.groups - 1));  // of one part
    const int parts = LPR / lanes, part = l / lanes;
    K marks[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      marks[j] = NONE;
      if (LPR * j >= a.groups) continue;
      const int g = (l & (lanes - 1)) + LPR * j;
      K m1 = NONE, m2 = NONE;
      if (g < a.groups) {
#pragma unroll 4
        for (int i = part; i < size; i += parts) {
          const K k = keys[g * (size + 1) + i];
          if (BY == BY_P) m2 = larger(smaller(k, m1), m2);
          m1 = larger(k, m1);
        }
      }
      for (int o = lanes; o < LPR; o <<= 1) {
        const K o1 = __shfl_xor(m1, o, 64);
        if constexpr (BY == BY_P) m2 = larger(smaller(o1, m1), larger(__shfl_xor(m2, o, 64), m2));
        m1 = larger(o1, m1);
      }
      if (a.best == 2 && m2 != NONE) m1 += m2;
      marks[j] = m1;
    }
    __builtin_amdgcn_wave_barrier();
    // A group stays if fewer than `keep` are above it (or level with it and before it).
    int above[SLOTS] = {};
    const int lane0 = threadIdx.x & 63 & ~(LPR - 1);
#pragma unroll 4
    for (int h = 0; h < a.groups; ++h) {
      K m = marks[0];
#pragma unroll
      for (int j = 1; j < SLOTS; ++j) m = h / LPR == j ? marks[j] : m;
      m = __shfl(m, lane0 + h % LPR, 64);
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) above[j] += m > marks[j] || (m == marks[j] && h < l + LPR * j);
    }
    uint64_t kept = 0;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) kept |= row_ballot<LPR>(above[j] < a.keep) << (LPR * j & 63);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (!((kept >> (group_of(i) & 63)) & 1)) key[i] = NONE;
  }
  ch[0] = ch[1] = -1;
  for (int n = 0; n < a.top; ++n) {
    K k1 = key[0];
#pragma unroll
    for (int i = 1; i < VPT; ++i) k1 = key[i] > k1 ? key[i] : k1;
    k1 = max_of<LPR>(k1);
    if (k1 == NONE) break;  // the same in all lanes of the row
    int at = 1 << 30;
#pragma unroll
    for (int i = VPT - 1; i >= 0; --i) at = key[i] == k1 ? l + LPR * i : at;
    at = min_of<LPR>(at);
#pragma unroll
    for (int i = 0; i < VPT; ++i) key[i] = at == l + LPR * i ? NONE : key[i];
    ch[0] = n == l ? at : ch[0];
    ch[1] = n == l + LPR ? at : ch[1];
  }
  double w[2] = {0.0, 0.0}, total = 0.0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (LPR * j >= a.top) break;
    const int64_t at = row * a.ldx + max(ch[j], 0);
    const double v = a.dtype == DT_F32 ? load1<DT_F32>(a.x, at) : a.dtype == DT_BF16 ? load1<DT_BF16>(a.x, at) : load1<DT_F16>(a.x, at);
    w[j] = SOFT ? exp_d(v - base) * per : 1.0 / (1.0 + exp_d(-v));
    w[j] = ch[j] >= 0 ? w[j] : 0.0;
    total += w[j];
  }
  if (a.renorm) {
    total = sum_of<LPR>(total);
    const double by = total > 0.0 ? total : 1.0;
#pragma unroll
    for (int j = 0; j < 2; ++j) w[j] = w[j] / by;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) wt[j] = bad ? bits_f(0x7FC00000u) : (float)(w[j] * a.scale);
}

// Weights and choices of a row, stored; its choices counted in LDS.
template <int LPR>
__device__ __forceinline__ void store_row(const RouteArgs& a, int64_t row, int l, const int ch[2], const float wt[2],
                                          int* s_count) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = l + LPR * j;
    if (n >= a.top) continue;
    a.weights[row * a.top + n] = wt[j];
    a.chosen[row * a.top + n] = ch[j];
    if (ch[j] >= 0) atomicAdd(&s_count[ch[j]], 1);
  }
}

// Counts of a block are a row of 4-aligned length.
__device__ __forceinline__ int count_pitch(int experts) { return (experts + 3) & ~3; }

// Where the keys of a thread's row are in LDS, a row for each LPR threads.  (The last two take rows apart.)
__device__ __forceinline__ void* row_keys(const RouteArgs& a, int* s_keys, int lpr) {
  return s_keys + (threadIdx.x / lpr) * 2 * (a.experts + a.groups + 2);
}

template <int LPR, int VPT, int BY, bool SOFT, bool GROUPS>
__global__ __launch_bounds__(1024) void k_route_select(RouteArgs a, int rows) {
  extern __shared__ __attribute__((aligned(16))) int s_count[];
  const int pitch = count_pitch(a.experts);
  for (int e = threadIdx.x; e < pitch; e += blockDim.x) s_count[e] = 0;
  __syncthreads();
  const int l = threadIdx.x % LPR;
  for (int r = threadIdx.x / LPR; r < rows; r += blockDim.x / LPR) {
    const int64_t row = (int64_t)blockIdx.x * rows + r;
    if (__builtin_amdgcn_readfirstlane((int)(row < a.rows)) == 0) break;  // the wave's first row, then all
    int ch[2];
    float wt[2];
    route_row<LPR, VPT, BY, SOFT, GROUPS>(a, min(row, a.rows - 1), l, row_keys(a, s_count + pitch, LPR), ch, wt);
    if (row < a.rows) store_row<LPR>(a, row, l, ch, wt, s_count);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < pitch; e += blockDim.x) a.counts[(int64_t)blockIdx.x * pitch + e] = s_count[e];
}

// Exclusive sums of s_off[0..E) in place, their total in s_off[E]; by one wave.
__device__ __forceinline__ void offsets_of(int* s_off, int E) {
  const int lane = threadIdx.x & 63;
  int run = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const int c = e < E ? s_off[e] : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(inc, o, 64);
      if (lane >= o) inc += u;
    }
    if (e < E) s_off[e] = run + inc - c;
    run += __shfl(inc, 63, 64);
  }
  if (lane == 0) s_off[E] = run;
}

// Choices [first, last) of a workgroup: its waves take consecutive pieces, a lane up to four of them, 64
// apart.  e: their experts (-1: none); rank: how many of the wave's choices before go to the
// same; s_wave [waves][E], zero before, holds the waves' counts afterwards.
constexpr int PLACE_PER = 4;
struct Choices {
  int64_t at[PLACE_PER];
  int e[PLACE_PER], rank[PLACE_PER];
};
__device__ __forceinline__ void load_choices(const RouteArgs& a, int64_t first, int64_t last, Choices& c) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t each = ((last - first + waves - 1) / waves + 63) / 64 * 64;
#pragma unroll
  for (int j = 0; j < PLACE_PER; ++j) {
    const int64_t at = first + each * wave + 64 * j + lane;
    c.at[j] = 64 * j < each && at < last ? at : -1;
    c.e[j] = c.at[j] >= 0 ? a.chosen[at] : -1;
  }
}
__device__ __forceinline__ void rank_choices(int E, Choices& c, int* s_wave) {
  const int lane = threadIdx.x & 63;
  int* mine = s_wave + (threadIdx.x >> 6) * E;
#pragma unroll
  for (int j = 0; j < PLACE_PER; ++j) {
    const int e = c.e[j];
    uint64_t same = __ballot(e >= 0);
    if (!same) continue;
    // The lanes with this lane's expert.
    for (int bit = 0; (1 << bit) < E; ++bit) {
      const uint64_t m = __ballot((e >> bit) & 1);
      same &= ((e >> bit) & 1) ? m : ~m;
    }
    const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
    int old = 0;
    if (e >= 0 && before == 0) old = atomicAdd(&mine[e], __builtin_popcountll(same));
    old = __shfl(old, e >= 0 ? __builtin_ctzll(same) : 0, 64);
    c.rank[j] = old + before;
  }
}
// The waves' counts to where each wave's first choice of an expert goes; s_next: the workgroup's first,
// afterwards the next one's.
__device__ __forceinline__ void start_waves(int E, int* s_next, int* s_wave) {
  const int waves = blockDim.x >> 6;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int n = s_next[e];
#pragma unroll 4
    for (int w = 0; w < waves; ++w) {
      const int c = s_wave[w * E + e];
      s_wave[w * E + e] = n;
      n += c;
    }
    s_next[e] = n;
  }
}
__device__ __forceinline__ void store_places(const RouteArgs& a, const Choices& c, const int* s_wave) {
  const int* mine = s_wave + (threadIdx.x >> 6) * a.experts;
#pragma unroll
  for (int j = 0; j < PLACE_PER; ++j) {
    if (c.at[j] < 0) continue;
    const int e = c.e[j];
    const int to = e >= 0 ? mine[e] + c.rank[j] : -1;
    a.place[c.at[j]] = to;
    if (e >= 0) a.row_of[to] = (int)((unsigned)c.at[j] / (unsigned)a.top);
  }
}

// Places of choices [first, last) in tiles of four a lane; c: the first tile's, ranked already.
__device__ __forceinline__ void place_tiles(const RouteArgs& a, int64_t first, int64_t last, Choices& c, int* s_next, int* s_wave) {
  const int tile = PLACE_PER * blockDim.x;
  for (;;) {
    __syncthreads();
    start_waves(a.experts, s_next, s_wave);
    __syncthreads();
    store_places(a, c, s_wave);
    first += tile;
    if (first >= last) return;
    load_choices(a, first, min(last, first + tile), c);
    __syncthreads();
    for (int e = threadIdx.x; e < ((int)blockDim.x >> 6) * a.experts; e += blockDim.x) s_wave[e] = 0;
    __syncthreads();
    rank_choices(a.experts, c, s_wave);
  }
}

// A block places the choices of `span` blocks of k_route_select (`rows` rows each), after adding up
// everyone's counts.
__global__ __launch_bounds__(1024) void k_route_place(RouteArgs a, int blocks, int rows, int span) {
  extern __shared__ int s_mem[];
  const int E = a.experts, pitch = count_pitch(E);
  int* s_next = s_mem;              // [pitch]: counts of the blocks before, then where the tile's first goes
  int* s_off = s_mem + pitch;       // [pitch + 4]
  int* s_wave = s_off + pitch + 4;  // [waves][E]
  const int tid = threadIdx.x, waves = blockDim.x >> 6;
  const int b0 = blockIdx.x * span;
  const int64_t total = a.rows * a.top;
  int64_t first = (int64_t)b0 * rows * a.top;
  const int64_t last = min(total, first + (int64_t)span * rows * a.top);
  Choices c;
  load_choices(a, first, min(last, first + PLACE_PER * (int64_t)blockDim.x), c);
  // Threads take four experts and every parts-th block.
  const int quads = pitch / 4, parts = max(1, (int)blockDim.x / quads);
  const int part = tid / quads, q = tid - part * quads;
  v4i before = v4i{}, all = v4i{};
  if (part < parts) {
#pragma unroll 8
    for (int b = part; b < blocks; b += parts) {
      const v4i n = *reinterpret_cast<const v4i*>(a.counts + (int64_t)b * pitch + 4 * q);
      before += b < b0 ? n : v4i{};
      all += n;
    }
  }
  for (int e = tid; e < 2 * pitch + 4 + waves * E; e += blockDim.x) s_mem[e] = 0;
  __syncthreads();
  if (part < parts) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      atomicAdd(&s_next[4 * q + i], before[i]);
      atomicAdd(&s_off[4 * q + i], all[i]);
    }
  }
  rank_choices(E, c, s_wave);
  __syncthreads();
  if (tid < 64) offsets_of(s_off, E);
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) s_next[e] += s_off[e];
  if (blockIdx.x == 0)
    for (int e = tid; e <= E; e += blockDim.x) a.offsets[e] = s_off[e];
  // Places that no choice takes, behind the last expert's rows.
  for (int64_t r = s_off[E] + (int64_t)blockIdx.x * blockDim.x + tid; r < total; r += (int64_t)gridDim.x * blockDim.x)
    a.row_of[r] = -1;
  place_tiles(a, first, last, c, s_next, s_wave);
}

// Few rows: choices, counts and places by one workgroup, in one launch.
template <int LPR, int VPT, int BY, bool SOFT, bool GROUPS>
__global__ __launch_bounds__(1024) void k_route_few(RouteArgs a) {
  extern __shared__ __attribute__((aligned(16))) int s_mem[];
  const int E = a.experts, pitch = count_pitch(E);
  int* s_off = s_mem;                 // [pitch + 4]
  int* s_wave = s_mem + pitch + 4;    // [waves][E], in waves * pitch
  int* s_keys = s_wave + ((int)blockDim.x >> 6) * pitch;
  for (int e = threadIdx.x; e < pitch + 4 + ((int)blockDim.x >> 6) * E; e += blockDim.x) s_mem[e] = 0;
  __syncthreads();
  const int l = threadIdx.x % LPR;
  for (int row = threadIdx.x / LPR; row < 64; row += blockDim.x / LPR) {
    if (__builtin_amdgcn_readfirstlane((int)(row < a.rows)) == 0) break;
    int ch[2];
    float wt[2];
    route_row<LPR, VPT, BY, SOFT, GROUPS>(a, min((int64_t)row, a.rows - 1), l, row_keys(a, s_keys, LPR), ch, wt);
    if (row < a.rows) store_row<LPR>(a, row, l, ch, wt, s_off);
  }
  __syncthreads();
  const int64_t all = a.rows * a.top;
  Choices c;
  load_choices(a, 0, min(all, PLACE_PER * (int64_t)blockDim.x), c);
  if (threadIdx.x < 64) offsets_of(s_off, E);
  rank_choices(E, c, s_wave);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += blockDim.x) a.offsets[e] = s_off[e];
  for (int64_t c2 = s_off[E] + threadIdx.x; c2 < all; c2 += blockDim.x) a.row_of[c2] = -1;
  place_tiles(a, 0, all, c, s_off, s_wave);
}

// out[i] = RNE(res[i] + gate * sum_j w[i, j] y[place[i, j]]): a thread owns eight elements of a row.
struct CombineArgs {
  const void* y;
  const int32_t* place;
  const float* w;
  const void* res;   // or nullptr
  const void* gate;  // or nullptr
  const int32_t* index;
  void* out;
  int64_t ldy, ldr, ldg, ldo;
  int64_t rows, y_rows, sets;
  unsigned per;  // rows of a set without an index
  int n, top, gate_f32;
};

template <int DT>
__device__ __forceinline__ void rows8(const void* p, int64_t at, int cnt, float* o) {
  if (cnt >= 8) {
    if constexpr (DT == DT_F32) {
      const v4f_el* q = reinterpret_cast<const v4f_el*>(reinterpret_cast<const float*>(p) + at);
      const v4f q0 = q[0], q1 = q[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = q0[i];
        o[4 + i] = q1[i];
      }
    } else {
      const u4v q = *reinterpret_cast<const u4v_el*>(reinterpret_cast<const uint16_t*>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) decode2<DT>(q[i], o[2 * i], o[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = i < cnt ? load1<DT>(p, at + i) : 0.0f;
  }
}

constexpr unsigned COMBINE_WIDE = 1u << 23;  // workgroups along x: a launch has less than 2^32 threads there

// TY: type of y; TO: of the residual and the output; gates in float32 or the 16-bit one of the two.  A
// wave has 512 elements of a row, so that the row's places and weights are scalars; four choices' rows
// are on their way at once.  Bound by the bytes of y, res and out: 17776 x 1920 of two choices with residual
// and gate 52.5 us = 5.2 TB/s, a large copy's rate (float32 y and out 102.7 us = 5.3); 4097 x 2047 of four, a tenth of
// them absent, rows at odd addresses, 22.8 us = 4.1 TB/s; eight rows 4.0 us.
template <int TY, int TO>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a, unsigned segments, unsigned items) {
  const unsigned item = (blockIdx.y * COMBINE_WIDE + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (item >= items) return;
  const int64_t row = item / segments;
  const int e = (int)(item % segments) * 512 + 8 * (threadIdx.x & 63);
  const int cnt = min(8, a.n - e);
  if (cnt <= 0) return;
  float r[8] = {};
  if (a.res) rows8<TO>(a.res, row * a.ldr + e, cnt, r);
  float v[8] = {};
  const int32_t* place = a.place + row * a.top;
  const float* weight = a.w + row * a.top;
  for (int j0 = 0; j0 < a.top; j0 += 4) {
    float q[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (j0 + u >= a.top) break;
      const int64_t at = place[j0 + u];
      if (at >= 0 && at < a.y_rows) {
        rows8<TY>(a.y, at * a.ldy + e, cnt, q[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[u][i] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (j0 + u >= a.top) break;
      const float w = weight[j0 + u];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] + q[u][i] * w;
    }
  }
  bool ok = true;
  if (a.gate) {
    const int64_t set = a.index ? a.index[row] : (unsigned)row / a.per;
    ok = set >= 0 && set < a.sets;
    float g[8];
    const int64_t ge = (ok ? set : 0) * a.ldg + e;
    if (a.gate_f32) rows8<DT_F32>(a.gate, ge, cnt, g);
    else rows8<TY == DT_F32 ? TO : TY>(a.gate, ge, cnt, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * g[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = !ok ? r[i] : a.res ? v[i] + r[i] : v[i];
  const int64_t o = row * a.ldo + e;
  if constexpr (TO == DT_F32) {
    float* p = reinterpret_cast<float*>(a.out) + o;
    if (cnt == 8) {
      reinterpret_cast<v4f_el*>(p)[0] = v4f{v[0], v[1], v[2], v[3]};
      reinterpret_cast<v4f_el*>(p)[1] = v4f{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < cnt) p[i] = v[i];
    }
  } else {
    u4v q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = cvt_pair<TO>(v[2 * i], v[2 * i + 1]);
    uint16_t* p = reinterpret_cast<uint16_t*>(a.out) + o;
    if (!ok && a.res) {  // the residual as it is, a NaN's bits too
      const uint16_t* rp = reinterpret_cast<const uint16_t*>(a.res) + row * a.ldr + e;
      q = cnt == 8 ? load8<false, false>(rp, 8) : load8<true, false>(rp, cnt);
    }
    if (cnt == 8) store8<false, false>(p, q, 8);
    else store8<true, false>(p, q, cnt);
  }
}

// Waves of a workgroup that places: its [waves][experts] counts within the 64 KiB of a launch without more.
static int place_waves(int experts) { return experts <= 512 ? 16 : 8; }
static size_t pitch_bytes(int experts) { return 4 * (size_t)((experts + 3) & ~3); }

template <int BY, bool SOFT, bool GROUPS>
static void launch_select(const RouteArgs& a, int blocks, int rows, hipStream_t st) {
  auto go = [&](auto lpr, auto vpt) {
    constexpr int L = decltype(lpr)::value, V = decltype(vpt)::value;
    const size_t pitch = pitch_bytes(a.experts);
    // Groups keep eight bytes an expert in LDS for each row at work: as many waves as 63 KiB hold beside
    // their counts.
    const size_t row = 8 * (size_t)(a.experts + a.groups + 2);
    const int fit = (int)((63 * 1024 - pitch - 16) / (pitch + 64 / L * row));
    const int most = a.groups > 1 ? 64 * std::max(1, std::min(16, fit)) : 1024;
    auto keys = [&](int block) { return a.groups > 1 ? (block / L) * row : (size_t)0; };
    if (!rows) {
      const int block = std::min(std::min(most, 64 * place_waves(a.experts)), ((int)a.rows * L + 63) / 64 * 64);
      hipLaunchKernelGGL((k_route_few<L, V, BY, SOFT, GROUPS>), dim3(1), dim3(block), pitch + 16 + (block / 64) * pitch + keys(block), st, a);
    } else {
      const int block = std::min(most, rows * L);
      hipLaunchKernelGGL((k_route_select<L, V, BY, SOFT, GROUPS>), dim3(blocks), dim3(block), pitch + keys(block), st, a, rows);
    }
  };
  const int e = a.experts;
  const std::integral_constant<int, 16> quarter;
  const std::integral_constant<int, 64> wave;
  if (e <= 16) go(quarter, std::integral_constant<int, 1>{});
  else if (e <= 32) go(quarter, std::integral_constant<int, 2>{});
  else if (e <= 64) go(quarter, std::integral_constant<int, 4>{});
  else if (e <= 96) go(quarter, std::integral_constant<int, 6>{});
  else if (e <= 128) go(quarter, std::integral_constant<int, 8>{});
  else if (e <= 160) go(quarter, std::integral_constant<int, 10>{});
  else if (e <= 192) go(quarter, std::integral_constant<int, 12>{});
  else if (e <= 256) go(quarter, std::integral_constant<int, 16>{});
  else if (e <= 512) go(wave, std::integral_constant<int, 8>{});
  else go(wave, std::integral_constant<int, 16>{});
}
template <int BY>
static void launch_select_by(const RouteArgs& a, int blocks, int rows, hipStream_t st) {
  if (a.softmax) {
    if (a.groups > 1) launch_select<BY, true, true>(a, blocks, rows, st);
    else launch_select<BY, true, false>(a, blocks, rows, st);
  } else {
    if (a.groups > 1) launch_select<BY, false, true>(a, blocks, rows, st);
    else launch_select<BY, false, false>(a, blocks, rows, st);
  }
}

// Rows of a block of k_route_select, 0 where one launch does all (in one pass of its workgroup, also where
// groups' keys fill LDS: 16 rows of 1024 experts in 64 groups take 86 us in one launch, 64 rows 36 in two;
// without groups 64 rows of 160 take 13 us in one and 14 in two).  Otherwise as many whole waves as leave
// the busiest compute unit the fewest rows, in one pass of a workgroup and no more than two workgroups a
// compute unit (k_route_place reads every one's counts) while rows are few enough for that; passes one after
// the other wait for each other's loads.
static int64_t wave_rows(int64_t experts) { return experts <= 256 ? 4 : 1; }
static int64_t most_select_blocks() { return 2 * (int64_t)vq_internal::persistent_blocks(); }
static int select_rows(int64_t rows, int64_t experts) {
  const int64_t wave = wave_rows(experts);
  if (rows <= (experts <= 64 ? 64 : 4 * wave)) return 0;
  const int64_t cus = vq_internal::persistent_blocks(), share = (rows + cus - 1) / cus;
  int64_t best = (share + 16 * wave - 1) / (16 * wave) * 16 * wave, cost = best + 1;
  for (int64_t r = wave; r <= 16 * wave; r += wave) {
    const int64_t blocks = (rows + r - 1) / r, c = (blocks + cus - 1) / cus * r;
    if (blocks > most_select_blocks() || c >= cost) continue;
    best = r;
    cost = c;
  }
  return (int)best;
}

}  // namespace vqk

namespace vq_internal {

using namespace vqk;

// A buffer made for a larger call has to do for a smaller one, which may be cut into more blocks: so many
// as no cut exceeds (blocks of a wave's rows or more, and at most most_select_blocks()).
int64_t route_experts_workspace_elems(int64_t rows, int64_t experts) {
  if (!select_rows(rows, experts)) return 0;
  const int64_t wave = wave_rows(experts);
  return std::min((rows + wave - 1) / wave, most_select_blocks()) * ((experts + 3) & ~3);
}

hipError_t launch_route_experts(const RouteExpertsParams& p, hipStream_t st) {
  RouteArgs a{};
  a.x = p.x;
  a.bias = p.bias;
  a.dtype = p.dtype;
  a.ldx = p.ldx;
  a.rows = p.rows;
  a.experts = p.experts;
  a.top = p.top;
  a.groups = p.groups;
  a.keep = p.keep;
  a.best = p.best;
  a.softmax = p.softmax;
  a.renorm = p.renorm;
  a.scale = p.scale;
  a.offsets = p.offsets;
  a.row_of = p.row_of;
  a.weights = p.weights;
  a.chosen = p.chosen;
  a.place = p.place;
  a.counts = p.counts;
  const int rows = select_rows(p.rows, p.experts);
  const int blocks = rows ? (int)((p.rows + rows - 1) / rows) : 0;
  if (p.rows) {
    if (a.bias || (a.groups > 1 && a.best == 2)) launch_select_by<BY_P>(a, blocks, rows, st);
    else launch_select_by<BY_SCORE>(a, blocks, rows, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !rows) return e;
  }
  // Blocks of choices for two or four a lane, where that many fit (without rows: zero offsets alone).
  const int span = std::max(1, 2048 / std::max(1, rows * p.top)), grid = std::max(1, (blocks + span - 1) / span);
  const int waves = place_waves(p.experts);
  const size_t lds = 2 * pitch_bytes(p.experts) + 16 + 4 * (size_t)waves * p.experts;
  hipLaunchKernelGGL(k_route_place, dim3(grid), dim3(64 * waves), lds, st, a, blocks, std::max(1, rows), span);
  return hipGetLastError();
}

hipError_t launch_combine(const CombineParams& p, hipStream_t st) {
  CombineArgs a{};
  a.y = p.y;
  a.place = p.place;
  a.w = p.weights;
  a.res = p.res;
  a.gate = p.mod.gate;
  a.index = p.mod.index;
  a.out = p.out;
  a.ldy = p.ldy;
  a.ldr = p.ldr;
  a.ldg = p.mod.ldg;
  a.ldo = p.ldo;
  a.rows = p.rows;
  a.y_rows = p.y_rows;
  a.sets = p.mod.sets;
  a.per = (unsigned)std::max<int64_t>(1, p.rows / p.mod.sets);
  a.n = (int)p.n;
  a.top = p.top;
  a.gate_f32 = p.mod.f32;
  const unsigned segments = (unsigned)((p.n + 511) / 512), items = (unsigned)p.rows * segments;  // below 2^32
  const unsigned blocks = items / 4 + (items % 4 != 0);
  const dim3 grid(std::min(blocks, COMBINE_WIDE), (blocks + COMBINE_WIDE - 1) / COMBINE_WIDE);
  auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(256), 0, st, a, segments, items); };
  if (p.y_dt == DT_F32) {
    if (p.out_dt == DT_F32) go(k_combine<DT_F32, DT_F32>);
    else if (p.out_dt == DT_BF16) go(k_combine<DT_F32, DT_BF16>);
    else go(k_combine<DT_F32, DT_F16>);
  } else if (p.y_dt == DT_BF16) {
    if (p.out_dt == DT_F32) go(k_combine<DT_BF16, DT_F32>);
    else go(k_combine<DT_BF16, DT_BF16>);
  } else {
    if (p.out_dt == DT_F32) go(k_combine<DT_F16, DT_F32>);
    else go(k_combine<DT_F16, DT_F16>);
  }
  return hipGetLastError();
}

}  // namespace vq_internal
