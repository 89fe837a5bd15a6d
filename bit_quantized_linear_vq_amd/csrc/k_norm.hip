// Root-mean-square norm with the residual's addition for gfx950: the rows that enter a
// linear layer, as 16-bit values or, quantized at once, as activation codes and scales.
//
//   h = RNE16(fl32(x + r))                      (h = x without a residual)
//   rstd = fl32(1 / sqrt(sum(h^2) / K + eps))   (the sum, division and root in float64)
//   v = fl32(fl32(h * rstd) * w)
//   y = RNE16(v), or the codes and scale of v as the row quantizer takes them from x
//
// The sum of squares is held in float64: the squares of 16-bit values are exact there, so
// rstd does not depend on the order of the sum (short of a tie at 2^-53) and the codes
// equal those of any other evaluation of the formula.
//
// Work layout: T threads own a row, each NP pieces of 8 elements that stay in registers
// from the load to the store, so x and r are read once and h, y or the codes written
// once; the kernel is bound by those bytes.  Piece j of thread t starts at element
// 8 (t + T j), one 16-byte access each (at any element's address: the hardware takes
// unaligned ones), contiguous over a wave.  With many rows a thread takes four pieces, so
// that up to 2048 elements a row needs one wave and no barrier; with few, one piece, for the
// latency.
//
// Measured, back to back over three sets of buffers: 17776 x 1920 with the residual, to codes 46.9 us = 5.1
// TB/s (alone in a trace 46.4-52, median 47.2), to 16 bits 45.5 us = 6.0 TB/s (50.8 over eight sets: the
// last-level cache holds the rest); 4113 x 4096 to 16 bits 27.2 us (21.4 over one set), 4113 x 4095 28.6 us;
// one row of 1920 4.5 us, 3.1 in a trace.  A large copy reaches 5.0-5.4 TB/s.
#include <algorithm>

#include "dev_common.h"
#include "gemm_common.h"
#include "rows_common.h"
#include "vq_internal.h"

namespace vqk {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;  // or nullptr
  const void* w;        // or nullptr: ones
  uint16_t* h;          // or nullptr
  uint16_t* y;
  int8_t* codes;
  float* scales;
  const int32_t* bits_dev;
  const int32_t* idx;
  const float* sgiven;  // static scales, or nullptr
  int64_t ldx, ldr, ldh, ldy;
  int64_t rows;
  double eps;
  int k, kp, w_f32, qbits, n_out, p1;
};

// What goes past the cache.  The sum, always: nobody reads it before the product has run (4113 x 4096
// to 16 bits 23.3 -> 21.6 us with buffers in use again, 8000 x 5760 to codes 69.7 -> 66.0; even also
// where the next call's residual is this one's sum).  x and the residual, read once, where the call's
// operands do not fit the last-level cache beside others: 17776 x 1920 to codes 49.1 -> 46.0 us, with the
// product that reads the codes, 1920 -> 5760, 254 -> 245; but what the layer before left in that cache
// should be found there (4113 x 4096 21.6, past it 26.0), and outlier channels are read twice.  Never what
// the product reads next: codes sent past it made 64 rows of 4096 with their product 19.6 -> 22.2 us.
//
// QUANT: codes and scales instead of y.  PAST: x and the residual past the cache.  T threads a row.
template <int DT, bool RES, bool QUANT, bool DUAL, int END, int NP, bool PAST = false>
__global__ __launch_bounds__(1024) void k_rmsnorm(NormArgs a, int T) {
  static_assert(END == END_WHOLE || !QUANT, "codes are written 8 at a time");
  constexpr bool TINY = END == END_TINY;
  static_assert(QUANT || !DUAL, "the outlier partition is one of codes");
  __shared__ double s_sum[2][16];
  __shared__ float s_max[2][16][2];
  __shared__ unsigned s_mask[DUAL ? 1024 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
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

  // Eight weights; a row's are read again with the row (they stay in the cache: kept in
  // registers they cost waves).
  auto weights = [&](int j, float* wv) {
    if (!a.w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) wv[i] = 1.0f;
      return;
    }
    const int e = at(j);
    if (TINY) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = min(i, a.k - 1);
        wv[i] = a.w_f32 ? reinterpret_cast<const float*>(a.w)[c] : load1<DT>(a.w, c);
      }
    } else if (a.w_f32) {
      const v4f_el* q = reinterpret_cast<const v4f_el*>(reinterpret_cast<const float*>(a.w) + e);
      const v4f w0 = q[0], w1 = q[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wv[i] = w0[i];
        wv[4 + i] = w1[i];
      }
    } else {
      const u4v q = *reinterpret_cast<const u4v_el*>(reinterpret_cast<const uint16_t*>(a.w) + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) decode2<DT>(q[i], wv[2 * i], wv[2 * i + 1]);
    }
  };
  // Whether one of this thread's weights is an infinity or NaN (the scales then say so: a
  // row maximum alone would pass a NaN by).
  bool w_bad = false;
  if constexpr (QUANT) {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      float wv[8];
      weights(j, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) z += wv[i] * 0.0f;
    }
    w_bad = !(z == 0.0f);
  }

  unsigned obits[NP] = {};
  int oidx[2] = {-1, -1};
  float ow[2] = {0.0f, 0.0f};
  if constexpr (DUAL) {
    for (int i = tid; i < 1024; i += blockDim.x) s_mask[i] = 0u;
    __syncthreads();
    for (int i = tid; i < a.n_out; i += blockDim.x) {
      const int o = a.idx[i];
      if (o >= 0 && o < a.k) atomicOr(&s_mask[o >> 5], 1u << (o & 31));
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int e = elem(j);
      if (e < a.k) obits[j] = (s_mask[e >> 5] >> (e & 31)) & 0xFFu;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = lt + 64 * i;
      if (lt < 64 && j < a.n_out) {
        const int o = a.idx[j];
        if (o >= 0 && o < a.k) {
          oidx[i] = o;
          ow[i] = !a.w ? 1.0f : a.w_f32 ? reinterpret_cast<const float*>(a.w)[o] : load1<DT>(a.w, o);
        }
      }
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
    const uint16_t* xr = a.x + rr * a.ldx;
    const uint16_t* sr = RES ? a.res + rr * a.ldr : nullptr;
    u4v raw[NP], rad[RES ? NP : 1];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      raw[j] = load8<TINY, PAST>(xr + at(j), a.k);
      if constexpr (RES) rad[j] = load8<TINY, PAST>(sr + at(j), a.k);
    }
    // The outlier channels' h, gathered before anyone stores h (h may be x or r itself).
    float ov[2] = {0.0f, 0.0f};
    if constexpr (DUAL) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (oidx[i] >= 0) {
          ov[i] = load1<DT>(xr, oidx[i]);
          if constexpr (RES) {
            float unused;
            decode2<DT>(cvt_pair<DT>(ov[i] + load1<DT>(sr, oidx[i]), 0.0f), ov[i], unused);
          }
          ov[i] = f32_fence(ov[i]);
        }
    }
    float v[NP][8];
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      if constexpr (RES) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x0, x1, r0, r1;
          decode2<DT>(raw[j][i], x0, x1);
          decode2<DT>(rad[j][i], r0, r1);
          raw[j][i] = cvt_pair<DT>(x0 + r0, x1 + r1);
        }
      }
      // Eight squares, each exact in float64; the pieces past the row's end repeat its first one.
      double p = 0.0;
      const int before = END == END_OVERLAP ? elem(j) - at(j) : 0;  // counted by the piece before
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        decode2<DT>(raw[j][i], v[j][2 * i], v[j][2 * i + 1]);
#pragma unroll
        for (int t = 2 * i; t < 2 * i + 2; ++t) {
          const float c = END == END_OVERLAP && t < before ? 0.0f : v[j][t];
          p = __builtin_fma((double)c, (double)c, p);
        }
      }
      ss += elem(j) < a.k ? p : 0.0;
    }
    ss = wave_sum_dpp(ss);
    if (wpr > 1) {
      if (lane == 0) s_sum[buf][wave] = ss;
      __syncthreads();
      ss = 0.0;
      for (int w = 0; w < wpr; ++w) ss += s_sum[buf][rib * wpr + w];
    }
    const float rstd = (float)(1.0 / sqrt(ss / kd + a.eps));

    if (a.h && row_ok) {
      uint16_t* hr = a.h + row * a.ldh;
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (elem(j) < a.k) store8<TINY, true>(hr + at(j), raw[j], a.k);
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      float wv[8];
      weights(j, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = (v[j][i] * rstd) * wv[i];
    }

    if constexpr (!QUANT) {
      if (row_ok) {
        uint16_t* yr = a.y + row * a.ldy;
#pragma unroll
        for (int j = 0; j < NP; ++j)
          if (elem(j) < a.k) {
            u4v o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = cvt_pair<DT>(v[j][2 * i], v[j][2 * i + 1]);
            store8<TINY, false>(yr + at(j), o, a.k);
          }
      }
    } else {
      if constexpr (DUAL) {
#pragma unroll
        for (int i = 0; i < 2; ++i) ov[i] = oidx[i] >= 0 ? (ov[i] * rstd) * ow[i] : 0.0f;
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((obits[j] >> i) & 1u) v[j][i] = 0.0f;
      }
      float r0 = rg[0], r1 = rg[1];
      const bool dynamic = !a.sgiven;
      if (dynamic) {
        float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          float pm = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) pm = fmaxf(pm, fabsf(v[j][i]));
          m0 = fmaxf(m0, elem(j) < a.k ? pm : 0.0f);
        }
        if (w_bad) m0 = bits_f(0x7F800000u);
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
        // A row with an infinity or NaN: its scales say so.
        if (!(rstd > 0.0f && rstd < bits_f(0x7F800000u)) || !(m0 < bits_f(0x7F800000u)) || !(m1 < bits_f(0x7F800000u))) {
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

template <int DT, bool RES, bool QUANT, bool DUAL, int END>
static void launch_norm_np(const NormArgs& a, int np, int grid, int block, int T, hipStream_t st) {
  switch (np) {
    case 1: hipLaunchKernelGGL((k_rmsnorm<DT, RES, QUANT, DUAL, END, 1>), dim3(grid), dim3(block), 0, st, a, T); break;
    case 2: hipLaunchKernelGGL((k_rmsnorm<DT, RES, QUANT, DUAL, END, 2>), dim3(grid), dim3(block), 0, st, a, T); break;
    default:
      // Above three quarters of the 256 MiB last-level cache: see above the kernel.
      if (!DUAL && a.rows * a.k * (2 + 2 * RES + 2 * (a.h != nullptr) + (QUANT ? 1 : 2)) > ((int64_t)192 << 20))
        hipLaunchKernelGGL((k_rmsnorm<DT, RES, QUANT, DUAL, END, 4, !DUAL>), dim3(grid), dim3(block), 0, st, a, T);
      else
        hipLaunchKernelGGL((k_rmsnorm<DT, RES, QUANT, DUAL, END, 4>), dim3(grid), dim3(block), 0, st, a, T);
      break;
  }
}

template <int DT, bool RES>
static void launch_norm_res(const NormArgs& a, bool quant, int np, int grid, int block, int T, hipStream_t st) {
  if (quant) {
    if (a.n_out) launch_norm_np<DT, RES, true, true, END_WHOLE>(a, np, grid, block, T, st);
    else launch_norm_np<DT, RES, true, false, END_WHOLE>(a, np, grid, block, T, st);
  } else if (a.k % 8 == 0) {
    launch_norm_np<DT, RES, false, false, END_WHOLE>(a, np, grid, block, T, st);
  } else if (a.k > 8) {
    launch_norm_np<DT, RES, false, false, END_OVERLAP>(a, np, grid, block, T, st);
  } else {
    hipLaunchKernelGGL((k_rmsnorm<DT, RES, false, false, END_TINY, 1>), dim3(grid), dim3(block), 0, st, a, T);
  }
}

template <int DT>
static void launch_norm_dt(const NormArgs& a, bool quant, int np, int grid, int block, int T, hipStream_t st) {
  if (a.res) launch_norm_res<DT, true>(a, quant, np, grid, block, T, st);
  else launch_norm_res<DT, false>(a, quant, np, grid, block, T, st);
}

}  // namespace vqk

namespace vq_internal {

using namespace vqk;

int norm_max_k() { return 1024 * 8 * 4; }

hipError_t launch_norm(const NormParams& p, hipStream_t st) {
  NormArgs a{};
  a.x = reinterpret_cast<const uint16_t*>(p.x);
  a.res = reinterpret_cast<const uint16_t*>(p.res);
  a.w = p.w;
  a.h = reinterpret_cast<uint16_t*>(p.h);
  a.y = reinterpret_cast<uint16_t*>(p.y);
  a.codes = p.codes;
  a.scales = p.scales;
  a.bits_dev = p.bits_dev;
  a.idx = p.idx;
  a.sgiven = p.static_scale;
  a.ldx = p.ldx;
  a.ldr = p.ldr;
  a.ldh = p.ldh;
  a.ldy = p.ldy;
  a.rows = p.rows;
  a.eps = p.eps;
  a.k = (int)p.k;
  a.kp = (int)p.kp;
  a.w_f32 = p.w_f32;
  a.qbits = p.bits;
  a.n_out = p.n_out;
  a.p1 = p.p1;
  const bool quant = p.codes != nullptr;
  // Pieces per thread and threads per row: four pieces with rows enough for every compute
  // unit's waves, else one (two or four where 1024 threads are not enough).
  const int pieces = (int)((p.k + 7) / 8);
  const int per = p.rows >= 1024 ? 4 : 1;
  const int T = std::min(1024, (pieces + 64 * per - 1) / (64 * per) * 64);
  const int each = (pieces + T - 1) / T;
  const int np = each <= 1 ? 1 : each <= 2 ? 2 : 4;
  const int block = T <= 128 ? 256 : T;
  const int64_t need = (p.rows + block / T - 1) / (block / T);
  // Workgroups of 32 waves per compute unit in all, two times what fits at once: 17776 x 1920 with
  // residual and codes 46.0 us (8: 53.1, 16: 46.9, 64: 45.8), without the residual 28.4 (30.7, 27.2, 30.4),
  // 8000 x 5760 61.7 (70.3, 71.7, 62.2).
  const int64_t most = (int64_t)persistent_blocks() * 32 / (block / 64);
  const int grid = (int)std::min(need, most);
  if (p.dtype == DT_BF16) launch_norm_dt<DT_BF16>(a, quant, np, grid, block, T, st);
  else launch_norm_dt<DT_F16>(a, quant, np, grid, block, T, st);
  return hipGetLastError();
}

}  // namespace vq_internal
