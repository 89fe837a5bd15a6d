// Norms before and after a block for gfx950: what stands between the last product of one block
// and the first of the next, in one pass over the rows.
//
//   u = y, or fl32(fl32(fl32(y - mean_y) * rstd_y) * pw)      (the branch's own norm)
//   s = RNE16(fl32(h + fl32(u * fl32(g * alpha))))            (gate and residual scale; s = h without a branch)
//   v = fl32(fl32(fl32(s - mean_s) * rstd_s) * w)
//   v = fl32(fl32(v * fl32(1 + c)) + d)                       (scale and shift)
//   n = RNE16(v), or the codes and scale of v as the row quantizer takes them
// with mean = fl32(sum x / K) for a layer norm and 0 for a root-mean-square one, and
// rstd = fl32(1 / sqrt(sum x^2 / K - (sum x / K)^2 + eps)).
//
// Sums, moments, division and root are float64: a 16-bit value and its square are exact there, and a
// sum of them loses at most some 2^-53 of its terms' size.  A layer norm's variance is (K S2 - S1^2) / K^2 of one pass's
// sums, both products in two parts: rounded (or as S2 / K - mean^2) their difference keeps only 2^-53
// (mean / deviation)^2 of itself, tens of float32 steps for fp16 rows of which one or two elements differ.  Nothing
// else is lost: in a row without an element below 2^-7 of its largest the sums are exact (squares of 11-bit values, 2^15
// of them, within 53 bits), and in any other the square of the mean is at most about 2 K times the variance.
// The float32 statistics, and with them the codes, do not depend on the order of the sums.
//
// Work layout as in the norm of one sum: T threads own a row, each NP pieces of 8 elements that
// stay in registers from the load to the store, so that y and h are read once and s, n or the
// codes written once; the kernel is bound by those bytes.  They stay there in 16 bits and are decoded
// where they are used, and parameters are read again with each row: held in float32 over the loop they
// took 160 registers and spilled (17776 x 1920 85 us).
//
// Measured, three sets of buffers in turn: 17776 x 1920, layer norm, the branch's own norm, a gate, scale and
// shift in float32 for each of 16 frames, to 16 bits 61.5 us = 4.4 TB/s (a large copy reaches 5.2); 4113 x
// 4096 with an index, to codes, 31.9 us = 3.7 TB/s; 17776 x 1920 without a branch 28.8 us; one row of 1920 4.1 us.
// A row of 1920 takes its wave 1222 vector instructions, about a quarter of them in float64: at least 35 of the 61.5 us are
// their issue, not waiting.  Tried and not kept: rows
// next to each other for one workgroup (modulation then stays in the first cache; 68 -> 76 us, 31 -> 35),
// two pieces a thread (62 -> 75 us, 31 -> 33), more waves by fewer registers (five waves a SIMD 62 -> 65, six
// 92: spills).
#include <algorithm>

#include "dev_common.h"
#include "gemm_common.h"
#include "rows_common.h"
#include "vq_internal.h"

namespace vqk {

enum : int { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };
enum : int { BR_NONE = 0, BR_PLAIN = 1, BR_NORMED = 2 };  // no branch, a branch, a branch with its own norm

struct GatedArgs {
  const uint16_t* y;  // or nullptr: no branch
  const uint16_t* h;
  const void* pw;  // or nullptr: ones
  const void* w;   // or nullptr: ones
  const void* gate;
  const void* sc;
  const void* sh;
  const int32_t* index;
  uint16_t* s;
  uint16_t* n;
  int8_t* codes;
  float* scales;
  const int32_t* bits_dev;
  const int32_t* idx;
  const float* sgiven;
  int64_t ldy, ldh, lds, ldn, ldg, ldsc, ldsh;
  int64_t rows, sets;
  double eps;
  unsigned per;  // rows of a set without an index (rows < 2^31)
  float alpha;
  int k, kp, pw_f32, w_f32, mod_f32, post, norm, qbits, n_out, p1;
};

// Eight parameters from element e of a row of float32 or 16-bit values (TINY: only the first k exist).
template <int DT, bool TINY>
__device__ __forceinline__ void params8(const void* p, int f32, int64_t e, int k, float* o) {
  if constexpr (TINY) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = e + min(i, k - 1);
      o[i] = f32 ? reinterpret_cast<const float*>(p)[c] : load1<DT>(p, c);
    }
  } else if (f32) {
    const v4f_el* q = reinterpret_cast<const v4f_el*>(reinterpret_cast<const float*>(p) + e);
    const v4f q0 = q[0], q1 = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = q0[i];
      o[4 + i] = q1[i];
    }
  } else {
    const u4v q = *reinterpret_cast<const u4v_el*>(reinterpret_cast<const uint16_t*>(p) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) decode2<DT>(q[i], o[2 * i], o[2 * i + 1]);
  }
}
template <int DT>
__device__ __forceinline__ float param1(const void* p, int f32, int64_t e) {
  return f32 ? reinterpret_cast<const float*>(p)[e] : load1<DT>(p, e);
}

// BR: the branch.  QUANT: codes and scales instead of n.  PAST: y and h past the cache.  T threads a row.
template <int DT, int BR, bool QUANT, bool DUAL, int END, int NP, bool PAST = false>
__global__ __launch_bounds__(1024) void k_gated_norm(GatedArgs a, int T) {
  static_assert(END == END_WHOLE || !QUANT, "codes are written 8 at a time");
  static_assert(QUANT || !DUAL, "the outlier partition is one of codes");
  constexpr bool TINY = END == END_TINY;
  __shared__ double s_sum[2][2][16][2];
  __shared__ float s_max[2][16][2];
  __shared__ unsigned s_mask[DUAL ? 1024 : 1];
  // A wave has one row: what goes by the row is the same for its lanes, and kept in scalar registers.
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wpr = T >> 6;  // waves per row
  const int rpb = (int)blockDim.x / T;
  const int rib = wave / wpr;
  const int lt = tid - rib * T;
  auto elem = [&](int j) { return 8 * (lt + T * j); };
  // Where piece j is read and written (a piece past the row's end reads its first one).
  auto at = [&](int j) {
    const int e = elem(j) < a.k ? elem(j) : 0;
    return END == END_OVERLAP ? min(e, a.k - 8) : e;
  };

  unsigned obits[NP] = {};
  int oidx[2] = {-1, -1};
  if constexpr (DUAL) {
    for (int i = tid; i < 1024; i += blockDim.x) s_mask[i] = 0u;
    __syncthreads();
    for (int i = tid; i < a.n_out; i += blockDim.x) {
      const int o = a.idx[i];
      if (o >= 0 && o < a.k) atomicOr(&s_mask[o >> 5], 1u << (o & 31));
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NP; ++j)
      if (elem(j) < a.k) obits[j] = (s_mask[elem(j) >> 5] >> (elem(j) & 31)) & 0xFFu;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lt < 64 && lt + 64 * i < a.n_out) {
        const int o = a.idx[lt + 64 * i];
        if (o >= 0 && o < a.k) oidx[i] = o;
      }
  }
  float qf = 0.0f, rg[2] = {0.0f, 0.0f};
  if constexpr (QUANT) {
    int b = a.bits_dev ? *a.bits_dev : a.qbits;
    b = (b == 4 || b == 6) ? b : 8;
    qf = (float)((1 << (b - 1)) - 1);
    if (a.sgiven) {
      for (int p = 0; p < (DUAL ? 2 : 1); ++p) {
        const float s = a.sgiven[p];
        rg[p] = 1.0f / s;
        if (!(s != 0.0f) || __builtin_isinf(rg[p])) rg[p] = 0.0f;
        if (blockIdx.x == 0 && tid == 0) a.scales[p] = s;
      }
    }
  }
  const double kd = (double)a.k;

  int buf = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < a.rows; row0 += (int64_t)gridDim.x * rpb, buf ^= 1) {
    const int64_t row = row0 + rib;
    const bool row_ok = row < a.rows;
    const int64_t rr = row_ok ? row : a.rows - 1;
    const uint16_t* hr = a.h + rr * a.ldh;
    const uint16_t* yr = BR ? a.y + rr * a.ldy : nullptr;
    u4v raw[NP], rad[BR ? NP : 1];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      raw[j] = load8<TINY, PAST>(hr + at(j), a.k);
      if constexpr (BR != BR_NONE) rad[j] = load8<TINY, PAST>(yr + at(j), a.k);
    }
    // The row's set of modulation rows; one outside them leaves the row without gate's branch, scale and shift.
    const int64_t set = a.index ? a.index[rr] : (unsigned)rr / a.per;
    const bool set_ok = set >= 0 && set < a.sets;
    const int64_t st = set_ok ? set : 0;
    // Parameters are read again with each row (they stay in the cache); moved out of the loop they
    // would be held in registers, which cost waves.
    const void *pw = a.pw, *wt = a.w;
    asm volatile("" : "+s"(pw), "+s"(wt));
    // The outlier channels' h and y, gathered before anyone stores s (s may be h or y itself).
    float oh[2] = {0.0f, 0.0f}, oy[2] = {0.0f, 0.0f};
    if constexpr (DUAL) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (oidx[i] >= 0) {
          oh[i] = f32_fence(load1<DT>(hr, oidx[i]));
          if constexpr (BR != BR_NONE) oy[i] = f32_fence(load1<DT>(yr, oidx[i]));
        }
    }

    // Sum and sum of squares over the row; the pieces past the row's end repeat its first one.  The
    // values stay in 16 bits and are decoded again where they are used: in float32 they cost registers,
    // and with them waves.
    auto moments = [&](const u4v (&q)[NP], int which, int kind, float& mean, float& rstd) {
      double s1 = 0.0, s2 = 0.0;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        double p1 = 0.0, p2 = 0.0;
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) decode2<DT>(q[j][i], v[2 * i], v[2 * i + 1]);
        const int before = END == END_OVERLAP ? elem(j) - at(j) : 0;  // counted by the piece before
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = TINY ? i < a.k : END == END_OVERLAP ? i >= before : true;
          const double c = in ? (double)v[i] : 0.0;
          p1 += c;
          p2 = __builtin_fma(c, c, p2);
        }
        s1 += elem(j) < a.k ? p1 : 0.0;
        s2 += elem(j) < a.k ? p2 : 0.0;
      }
      s2 = wave_sum_dpp(s2);
      if (kind == NORM_LAYER) s1 = wave_sum_dpp(s1);
      if (wpr > 1) {
        if (lane == 0) {
          s_sum[buf][which][wave][0] = s1;
          s_sum[buf][which][wave][1] = s2;
        }
        __syncthreads();
        s1 = s2 = 0.0;
        for (int w = 0; w < wpr; ++w) {
          s1 += s_sum[buf][which][rib * wpr + w][0];
          s2 += s_sum[buf][which][rib * wpr + w][1];
        }
      }
      double var = s2 / kd;
      mean = 0.0f;
      if (kind == NORM_LAYER) {
        const double q = kd * s2, p = s1 * s1;
        var = ((q - p) + (__builtin_fma(kd, s2, -q) - __builtin_fma(s1, s1, -p))) / (kd * kd);
        // (NaN stays: max would take it away)
        var = var < 0.0 ? 0.0 : var;
        mean = (float)(s1 / kd);
      }
      rstd = (float)(1.0 / sqrt(var + a.eps));
    };

    float pmean = 0.0f, prstd = 0.0f;
    if constexpr (BR == BR_NORMED) moments(rad, 0, a.post, pmean, prstd);
    if constexpr (BR != BR_NONE) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        float p[8], g[8];
        if (BR == BR_NORMED && pw) params8<DT, TINY>(pw, a.pw_f32, at(j), a.k, p);
        if (a.gate) params8<DT, TINY>(a.gate, a.mod_f32, st * a.ldg + at(j), a.k, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u[2], x[2];
          asm volatile("" : "+v"(rad[j][i]));  // decoded anew, not kept from the moments
          decode2<DT>(rad[j][i], u[0], u[1]);
          decode2<DT>(raw[j][i], x[0], x[1]);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if constexpr (BR == BR_NORMED) {
              u[t] = (u[t] - pmean) * prstd;
              if (pw) u[t] = u[t] * p[2 * i + t];
            }
            const float ga = a.gate ? g[2 * i + t] * a.alpha : a.alpha;
            u[t] = x[t] + u[t] * ga;
          }
          const unsigned sum = cvt_pair<DT>(u[0], u[1]);
          raw[j][i] = set_ok ? sum : raw[j][i];  // h as it is, a NaN's bits too
        }
      }
    }
    float mean, rstd;
    moments(raw, 1, a.norm, mean, rstd);

    if (BR != BR_NONE && row_ok) {
      uint16_t* sr = a.s + row * a.lds;
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (elem(j) < a.k) store8<TINY, true>(sr + at(j), raw[j], a.k);
    }
    // Piece j of the output before its last rounding.
    auto normed = [&](int j, float (&v)[8]) {
      float p[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x0, x1;
        asm volatile("" : "+v"(raw[j][i]));  // decoded anew, as above
        decode2<DT>(raw[j][i], x0, x1);
        v[2 * i] = (x0 - mean) * rstd;
        v[2 * i + 1] = (x1 - mean) * rstd;
      }
      if (wt) {
        params8<DT, TINY>(wt, a.w_f32, at(j), a.k, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * p[i];
      }
      if (a.sc && set_ok) {
        params8<DT, TINY>(a.sc, a.mod_f32, st * a.ldsc + at(j), a.k, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * (1.0f + p[i]);
      }
      if (a.sh && set_ok) {
        params8<DT, TINY>(a.sh, a.mod_f32, st * a.ldsh + at(j), a.k, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] + p[i];
      }
    };

    if constexpr (!QUANT) {
      if (row_ok) {
        uint16_t* nr = a.n + row * a.ldn;
#pragma unroll
        for (int j = 0; j < NP; ++j)
          if (elem(j) < a.k) {
            float v[8];
            normed(j, v);
            u4v o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = cvt_pair<DT>(v[2 * i], v[2 * i + 1]);
            store8<TINY, false>(nr + at(j), o, a.k);
          }
      }
    } else {
      float v[NP][8];
#pragma unroll
      for (int j = 0; j < NP; ++j) normed(j, v[j]);
      float ov[2] = {0.0f, 0.0f};
      // A value that is an infinity or NaN: the row's scales say so (a maximum alone would pass a NaN by).
      float bad = 0.0f;
      if constexpr (DUAL) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (oidx[i] >= 0) {
            const int o = oidx[i];
            float x = oh[i];
            if constexpr (BR != BR_NONE) {
              float u = oy[i];
              if constexpr (BR == BR_NORMED) {
                u = (u - pmean) * prstd;
                if (a.pw) u = u * param1<DT>(a.pw, a.pw_f32, o);
              }
              const float ga = a.gate ? param1<DT>(a.gate, a.mod_f32, st * a.ldg + o) * a.alpha : a.alpha;
              u = set_ok ? x + u * ga : x;
              float unused;
              decode2<DT>(cvt_pair<DT>(u, 0.0f), x, unused);
            }
            x = (x - mean) * rstd;
            if (a.w) x = x * param1<DT>(a.w, a.w_f32, o);
            if (a.sc && set_ok) x = x * (1.0f + param1<DT>(a.sc, a.mod_f32, st * a.ldsc + o));
            if (a.sh && set_ok) x = x + param1<DT>(a.sh, a.mod_f32, st * a.ldsh + o);
            ov[i] = x;
            bad += x * 0.0f;
          }
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((obits[j] >> i) & 1u) v[j][i] = 0.0f;
      }
      float r0 = rg[0], r1 = rg[1];
      if (!a.sgiven) {
        float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          float pm = 0.0f, pb = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            pm = fmaxf(pm, fabsf(v[j][i]));
            pb = __builtin_fmaf(v[j][i], 0.0f, pb);
          }
          m0 = fmaxf(m0, elem(j) < a.k ? pm : 0.0f);
          bad += elem(j) < a.k ? pb : 0.0f;
        }
        if (!(bad == 0.0f)) m0 = bits_f(0x7F800000u);
        m0 = wave_max(m0);
        if constexpr (DUAL) m1 = wave_max(fmaxf(fabsf(ov[0]), fabsf(ov[1])));
        if (wpr > 1) {
          if (lane == 0) {
            s_max[buf][wave][0] = m0;
            s_max[buf][wave][1] = m1;
          }
          __syncthreads();
          for (int w = 0; w < wpr; ++w) {
            m0 = fmaxf(m0, s_max[buf][rib * wpr + w][0]);
            if constexpr (DUAL) m1 = fmaxf(m1, s_max[buf][rib * wpr + w][1]);
          }
        }
        float s0, s1 = 0.0f;
        dyn_scale(m0, qf, r0, s0);
        if constexpr (DUAL) dyn_scale(m1, qf, r1, s1);
        if (!(m0 < bits_f(0x7F800000u)) || !(m1 < bits_f(0x7F800000u))) {
          r0 = r1 = 0.0f;
          s0 = s1 = bits_f(0x7FC00000u);
        }
        if (row_ok && lt == 0) {
          a.scales[row * (DUAL ? 2 : 1)] = s0;
          if constexpr (DUAL) a.scales[2 * row + 1] = s1;
        }
      }
      if (row_ok) {
        int8_t* cr = a.codes + row * a.kp;
#pragma unroll
        for (int j = 0; j < NP; ++j)
          if (elem(j) < a.k) {
            unsigned u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = qbyte(v[j][i], r0, qf);
            *reinterpret_cast<u2v*>(cr + elem(j)) =
                u2v{pack4_lo(u[0], u[1], u[2], u[3]), pack4_lo(u[4], u[5], u[6], u[7])};
          }
        if constexpr (DUAL) {
          if (lt < 64) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (lt + 64 * i < a.p1) cr[a.k + lt + 64 * i] = (int8_t)(qbyte(ov[i], r1, qf) & 0xFFu);
          }
        }
      }
    }
  }
}

template <int DT, int BR, bool QUANT, bool DUAL, int END>
static void launch_gated_np(const GatedArgs& a, int np, int grid, int block, int T, hipStream_t st) {
  switch (np) {
    case 1: hipLaunchKernelGGL((k_gated_norm<DT, BR, QUANT, DUAL, END, 1>), dim3(grid), dim3(block), 0, st, a, T); break;
    case 2: hipLaunchKernelGGL((k_gated_norm<DT, BR, QUANT, DUAL, END, 2>), dim3(grid), dim3(block), 0, st, a, T); break;
    default:
      // Read once, y and h go past the last-level cache where the call's operands take more than three
      // quarters of it (17776 x 1920 to 16 bits 70 -> 62 us; 4113 x 4096 to codes, which fit, 31 -> 34).
      // Outlier channels are read twice.
      if (!DUAL && a.rows * a.k * ((BR ? 6 : 2) + (QUANT ? 1 : 2)) > ((int64_t)192 << 20))
        hipLaunchKernelGGL((k_gated_norm<DT, BR, QUANT, DUAL, END, 4, !DUAL>), dim3(grid), dim3(block), 0, st, a, T);
      else
        hipLaunchKernelGGL((k_gated_norm<DT, BR, QUANT, DUAL, END, 4>), dim3(grid), dim3(block), 0, st, a, T);
      break;
  }
}

template <int DT, int BR>
static void launch_gated_br(const GatedArgs& a, int np, int grid, int block, int T, hipStream_t st) {
  if (a.codes) {
    if (a.n_out) launch_gated_np<DT, BR, true, true, END_WHOLE>(a, np, grid, block, T, st);
    else launch_gated_np<DT, BR, true, false, END_WHOLE>(a, np, grid, block, T, st);
  } else if (a.k % 8 == 0) {
    launch_gated_np<DT, BR, false, false, END_WHOLE>(a, np, grid, block, T, st);
  } else if (a.k > 8) {
    launch_gated_np<DT, BR, false, false, END_OVERLAP>(a, np, grid, block, T, st);
  } else {
    hipLaunchKernelGGL((k_gated_norm<DT, BR, false, false, END_TINY, 1>), dim3(grid), dim3(block), 0, st, a, T);
  }
}

template <int DT>
static void launch_gated_dt(const GatedArgs& a, int np, int grid, int block, int T, hipStream_t st) {
  if (!a.y) launch_gated_br<DT, BR_NONE>(a, np, grid, block, T, st);
  else if (a.post == NORM_NONE) launch_gated_br<DT, BR_PLAIN>(a, np, grid, block, T, st);
  else launch_gated_br<DT, BR_NORMED>(a, np, grid, block, T, st);
}

}  // namespace vqk

namespace vq_internal {

using namespace vqk;

hipError_t launch_gated_norm(const GatedNormParams& p, hipStream_t st) {
  GatedArgs a{};
  a.y = reinterpret_cast<const uint16_t*>(p.y);
  a.h = reinterpret_cast<const uint16_t*>(p.h);
  a.pw = p.pw;
  a.w = p.w;
  a.gate = p.mod.gate;
  a.sc = p.mod.scale;
  a.sh = p.mod.shift;
  a.index = p.mod.index;
  a.s = reinterpret_cast<uint16_t*>(p.s);
  a.n = reinterpret_cast<uint16_t*>(p.n);
  a.codes = p.codes;
  a.scales = p.scales;
  a.bits_dev = p.bits_dev;
  a.idx = p.idx;
  a.sgiven = p.static_scale;
  a.ldy = p.ldy;
  a.ldh = p.ldh;
  a.lds = p.lds;
  a.ldn = p.ldn;
  a.ldg = p.mod.ldg;
  a.ldsc = p.mod.ldsc;
  a.ldsh = p.mod.ldsh;
  a.rows = p.rows;
  a.sets = p.mod.sets;
  a.per = (unsigned)(p.rows / p.mod.sets);
  a.eps = p.eps;
  a.alpha = p.alpha;
  a.k = (int)p.k;
  a.kp = (int)p.kp;
  a.pw_f32 = p.pw_f32;
  a.w_f32 = p.w_f32;
  a.mod_f32 = p.mod.f32;
  a.post = p.post;
  a.norm = p.norm;
  a.qbits = p.bits;
  a.n_out = p.n_out;
  a.p1 = p.p1;
  // Pieces per thread and threads per row as in the norm of one sum: four pieces with rows enough
  // for every compute unit's waves, else one (two or four where 1024 threads are not enough).
  const int pieces = (int)((p.k + 7) / 8);
  const int per = p.rows >= 1024 ? 4 : 1;
  const int T = std::min(1024, (pieces + 64 * per - 1) / (64 * per) * 64);
  const int each = (pieces + T - 1) / T;
  const int np = each <= 1 ? 1 : each <= 2 ? 2 : 4;
  const int block = T <= 128 ? 128 : T;
  const int64_t need = (p.rows + block / T - 1) / (block / T);
  const int64_t most = (int64_t)persistent_blocks() * 64 / (block / 64);
  const int grid = (int)std::min(need, most);
  if (p.dtype == DT_BF16) launch_gated_dt<DT_BF16>(a, np, grid, block, T, st);
  else launch_gated_dt<DT_F16>(a, np, grid, block, T, st);
  return hipGetLastError();
}

}  // namespace vq_internal
