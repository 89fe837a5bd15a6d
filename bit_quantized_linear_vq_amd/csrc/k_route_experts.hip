// Routing to experts and back for gfx950: from the router's scores to rows sorted by expert (what
// the experts' products take), and from the experts' rows to their tokens again.
//
// Routing.  p = softmax or sigmoid of a row of scores; the choice goes by p + bias (by the scores
// themselves without a bias: the same order, with no rounding), in the groups whose best one or two
// sum highest; ties go to the lower index.  Whole numbers come out, so what they are compared by is
// float64: two values of p + bias may differ by less than float32 holds, and the exponentials are
// some tens of instructions against a launch.
//   k_route_select  a wave (or 16 of its lanes) a row: choices, weights, and the block's count for
//                   each expert
//   k_route_place   offsets, and each choice's place: rows before it in its expert's segment, by
//                   ascending token and choice.  Counts are whole numbers, so the order of their sums does not
//                   matter, and places are the same in every call.
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
  int experts, top, groups, keep, best, softmax, renorm;
  float scale;
  int32_t* offsets;
  int32_t* row_of;  // [rows * top]
  float* weights;   // [rows, top]
  int32_t* chosen;  // [rows, top]
  int32_t* place;   // [rows, top]
  int32_t* counts;  // [blocks, experts]
};

constexpr int ROUTE_ROWS = 64;   // rows of a block of k_route_select
constexpr double NONE = -__builtin_huge_val();

// The larger key, of equal ones that of the lower index, over LPR lanes (all of them get it).
template <int LPR>
__device__ __forceinline__ void best_of(double& key, int& at) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) {
    const double k2 = __shfl_xor(key, o, 64);
    const int a2 = __shfl_xor(at, o, 64);
    const bool take = k2 > key || (k2 == key && a2 < at);
    key = take ? k2 : key;
    at = take ? a2 : at;
  }
}
template <int LPR>
__device__ __forceinline__ double sum_of(double v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}
template <int LPR>
__device__ __forceinline__ double max_of(double v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v = fmax(v, __shfl_xor(v, o, 64));
  return v;
}
template <int LPR>
__device__ __forceinline__ bool any_of(bool b) {
  const int lane = threadIdx.x & 63;
  const uint64_t m = __ballot(b);
  return LPR == 64 ? m != 0 : ((m >> (lane & ~(LPR - 1))) & ((1ull << (LPR & 63)) - 1)) != 0;
}

// LPR lanes own a row, lane l the experts l + LPR i.
template <int DT, int LPR, int VPT>
__global__ __launch_bounds__(256) void k_route_select(RouteArgs a) {
  extern __shared__ int s_count[];
  for (int e = threadIdx.x; e < a.experts; e += 256) s_count[e] = 0;
  __syncthreads();
  const int l = threadIdx.x % LPR;
  for (int r = threadIdx.x / LPR; r < ROUTE_ROWS; r += 256 / LPR) {
    const int64_t row = (int64_t)blockIdx.x * ROUTE_ROWS + r;
    if (__builtin_amdgcn_readfirstlane((int)(row < a.rows)) == 0) break;  // the wave's first row, then all
    const bool row_ok = row < a.rows;
    const int64_t rr = row_ok ? row : a.rows - 1;
    double x[VPT], key[VPT];
    double top = NONE;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = l + LPR * i;
      x[i] = e < a.experts ? (double)load1<DT>(a.x, rr * a.ldx + e) : NONE;
      bad |= x[i] != x[i] || (a.softmax && x[i] == -NONE);
      top = fmax(top, x[i]);
    }
    // p in x's place
    double denom = 1.0;
    if (a.softmax) {
      top = max_of<LPR>(top);
      const double base = top == NONE ? 0.0 : top;
      denom = 0.0;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        key[i] = x[i];
        x[i] = exp(x[i] - base);
        denom += x[i];
      }
      denom = sum_of<LPR>(denom);
      denom = denom > 0.0 ? denom : 1.0;
#pragma unroll
      for (int i = 0; i < VPT; ++i) x[i] = x[i] / denom;
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        key[i] = x[i];
        x[i] = 1.0 / (1.0 + exp(-x[i]));
      }
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int e = l + LPR * i;
        if (e < a.experts) {
          const double k = x[i] + (double)a.bias[e];
          key[i] = key[i] == NONE ? NONE : k;
          bad |= key[i] != key[i];
        }
      }
    }
    bad = any_of<LPR>(bad);
#pragma unroll
    for (int i = 0; i < VPT; ++i) key[i] = bad ? NONE : key[i];
    if (a.groups > 1) {
      // Group after group its mark, then the groups that stay, then the others' keys away.
      const int size = a.experts / a.groups;
      const bool by_p = a.best == 2 && !a.bias;
      double mark = NONE;  // lane g of the row holds group g's, g + LPR the next one ..
      double marks[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) marks[j] = NONE;
      for (int g = 0; g < a.groups; ++g) {
        double k1 = NONE;
        int at = 1 << 30;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int e = l + LPR * i;
          if (e / size != g || e >= a.experts) continue;
          const double k = by_p && key[i] != NONE ? x[i] : key[i];
          if (k > k1) {
            k1 = k;
            at = e;
          }
        }
        best_of<LPR>(k1, at);
        mark = k1;
        if (a.best == 2 && size > 1) {
          double k2 = NONE;
#pragma unroll
          for (int i = 0; i < VPT; ++i) {
            const int e = l + LPR * i;
            if (e / size != g || e >= a.experts || e == at) continue;
            const double k = by_p && key[i] != NONE ? x[i] : key[i];
            k2 = fmax(k2, k);
          }
          k2 = max_of<LPR>(k2);
          mark += k2 == NONE ? 0.0 : k2;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (g == l + LPR * j) marks[j] = mark;
      }
      uint64_t kept = 0;
      for (int n = 0; n < a.keep; ++n) {
        double k1 = NONE;
        int at = 1 << 30;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int g = l + LPR * j;
          if (g < a.groups && !((kept >> g) & 1) && (marks[j] > k1 || at == 1 << 30)) {
            k1 = marks[j];
            at = g;
          }
        }
        best_of<LPR>(k1, at);
        kept |= 1ull << at;
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int e = l + LPR * i;
        if (e < a.experts && !((kept >> (e / size)) & 1)) key[i] = NONE;
      }
    }
    // Choice after choice; lane j of the row keeps choice j (and j + LPR).
    double w[2] = {0.0, 0.0}, total = 0.0;
    int ch[2] = {-1, -1};
    for (int n = 0; n < a.top; ++n) {
      double k1 = NONE;
      int at = 1 << 30;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (key[i] > k1) {
          k1 = key[i];
          at = l + LPR * i;
        }
      best_of<LPR>(k1, at);
      if (k1 == NONE) break;  // the same in all lanes of the row
      double p = 0.0;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (at == l + LPR * i) {
          p = x[i];
          key[i] = NONE;
        }
      p = sum_of<LPR>(p);
      total += p;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (n == l + LPR * j) {
          w[j] = p;
          ch[j] = at;
        }
    }
    if (row_ok) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = l + LPR * j;
        if (n >= a.top) continue;
        double v = a.renorm ? (total > 0.0 ? w[j] / total : 0.0) : w[j];
        if (bad) v = __builtin_nan("");
        a.weights[row * a.top + n] = (float)(v * (double)a.scale);
        a.chosen[row * a.top + n] = ch[j];
        if (ch[j] >= 0) atomicAdd(&s_count[ch[j]], 1);
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += 256) a.counts[(int64_t)blockIdx.x * a.experts + e] = s_count[e];
}

// A block places the choices of `span` blocks of k_route_select: its waves take consecutive pieces of
// them, count their experts, and go through them 64 at a time.
__global__ __launch_bounds__(1024) void k_route_place(RouteArgs a, int blocks, int span) {
  extern __shared__ int s_mem[];
  const int E = a.experts;
  int* s_base = s_mem;          // [E]: where this block's first choice of an expert goes
  int* s_off = s_mem + E;       // [E + 1]
  int* s_wave = s_off + E + 1;  // [waves][E]
  const int waves = blockDim.x >> 6;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b0 = blockIdx.x * span;
  for (int e = tid; e < E; e += blockDim.x) {
    int before = 0, all = 0;
    for (int b = 0; b < blocks; ++b) {
      const int c = a.counts[(int64_t)b * E + e];
      before += b < b0 ? c : 0;
      all += c;
    }
    s_base[e] = before;
    s_off[e] = all;
  }
  for (int i = tid; i < waves * E; i += blockDim.x) s_wave[i] = 0;
  __syncthreads();
  if (wave == 0) {
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
  __syncthreads();
  const int64_t all = a.rows * a.top;
  const int64_t first = (int64_t)b0 * ROUTE_ROWS * a.top;
  const int64_t last = min(all, first + (int64_t)span * ROUTE_ROWS * a.top);
  const int64_t each = (last - first + waves - 1) / waves;
  const int64_t w0 = min(last, first + each * wave), w1 = min(last, w0 + each);
  for (int64_t c = w0 + lane; c < w1; c += 64) {
    const int e = a.chosen[c];
    if (e >= 0) atomicAdd(&s_wave[wave * E + e], 1);
  }
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) {
    int at = s_off[e] + s_base[e];
    for (int w = 0; w < waves; ++w) {
      const int c = s_wave[w * E + e];
      s_wave[w * E + e] = at;
      at += c;
    }
  }
  __syncthreads();
  volatile int* mine = s_wave + wave * E;
  for (int64_t c0 = w0; c0 < w1; c0 += 64) {
    const int64_t c = c0 + lane;
    const int e = c < w1 ? a.chosen[c] : -1;
    // The lanes with this lane's expert.
    uint64_t same = __ballot(e >= 0);
    for (int bit = 0; (1 << bit) < E; ++bit) {
      const uint64_t m = __ballot((e >> bit) & 1);
      same &= ((e >> bit) & 1) ? m : ~m;
    }
    const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
    int at = -1;
    if (e >= 0) at = mine[e] + rank;
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && rank == 0) mine[e] = at + __builtin_popcountll(same);
    __builtin_amdgcn_wave_barrier();
    if (c < w1) {
      a.place[c] = at;
      if (e >= 0) a.row_of[at] = (int)(c / a.top);
    }
  }
  if (blockIdx.x == 0)
    for (int e = tid; e <= E; e += blockDim.x) a.offsets[e] = s_off[e];
  // Places that no choice takes, behind the last expert's rows.
  for (int64_t c = s_off[E] + (int64_t)blockIdx.x * blockDim.x + tid; c < all; c += (int64_t)gridDim.x * blockDim.x)
    a.row_of[c] = -1;
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
  int64_t rows, y_rows, sets, per;
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

// TY: type of y; TO: of the residual and the output; gates in float32 or TG.
template <int TY, int TO>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a, int pieces) {
  const int64_t total = a.rows * pieces;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
    const int64_t row = t / pieces;
    const int e = 8 * (int)(t - row * pieces);
    const int cnt = min(8, a.n - e);
    float v[8] = {};
    for (int j = 0; j < a.top; ++j) {
      const int64_t at = a.place[row * a.top + j];
      const float w = a.w[row * a.top + j];
      if (at >= 0 && at < a.y_rows) {
        float q[8];
        rows8<TY>(a.y, at * a.ldy + e, cnt, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] + q[i] * w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] + 0.0f * w;
      }
    }
    float r[8] = {};
    if (a.res) rows8<TO>(a.res, row * a.ldr + e, cnt, r);
    bool ok = true;
    if (a.gate) {
      const int64_t set = a.index ? a.index[row] : row / a.per;
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
      for (int i = 0; i < 8; ++i)
        if (i < cnt) p[i] = v[i];
    } else {
      u4v q;
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = cvt_pair<TO>(v[2 * i], v[2 * i + 1]);
      uint16_t* p = reinterpret_cast<uint16_t*>(a.out) + o;
      if (cnt == 8) store8<false, false>(p, q, 8);
      else store8<true, false>(p, q, cnt);
    }
  }
}

template <int DT>
static void launch_select(const RouteArgs& a, int blocks, hipStream_t st) {
  const size_t lds = 4 * (size_t)a.experts;
  auto go = [&](auto lpr, auto vpt) {
    hipLaunchKernelGGL((k_route_select<DT, decltype(lpr)::value, decltype(vpt)::value>), dim3(blocks), dim3(256), lds, st, a);
  };
  const int e = a.experts;
  if (e <= 16) go(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  else if (e <= 32) go(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
  else if (e <= 64) go(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  else if (e <= 128) go(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
  else if (e <= 256) go(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
  else if (e <= 512) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

}  // namespace vqk

namespace vq_internal {

using namespace vqk;

int64_t route_experts_blocks(int64_t rows) { return (rows + ROUTE_ROWS - 1) / ROUTE_ROWS; }

hipError_t launch_route_experts(const RouteExpertsParams& p, hipStream_t st) {
  RouteArgs a{};
  a.x = p.x;
  a.bias = p.bias;
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
  const int blocks = (int)route_experts_blocks(p.rows);
  if (blocks) {
    if (p.dtype == DT_F16) launch_select<DT_F16>(a, blocks, st);
    else if (p.dtype == DT_BF16) launch_select<DT_BF16>(a, blocks, st);
    else launch_select<DT_F32>(a, blocks, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int span = 4, grid = std::max(1, (blocks + span - 1) / span);
  // [waves][experts] counts within the 64 KiB of a launch without more
  const int waves = p.experts <= 512 ? 16 : 8;
  hipLaunchKernelGGL(k_route_place, dim3(grid), dim3(64 * waves), 4 * ((waves + 2) * (size_t)p.experts + 1), st, a, blocks, span);
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
  a.per = std::max<int64_t>(1, p.rows / p.mod.sets);
  a.n = (int)p.n;
  a.top = p.top;
  a.gate_f32 = p.mod.f32;
  const int pieces = (int)((p.n + 7) / 8);
  const int64_t need = (p.rows * pieces + 255) / 256;
  const int grid = (int)std::min<int64_t>(need, (int64_t)persistent_blocks() * 16);
  auto go = [&](auto k) { hipLaunchKernelGGL(k, dim3(grid), dim3(256), 0, st, a, pieces); };
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
