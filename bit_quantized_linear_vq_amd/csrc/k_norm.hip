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
// 8 (t + T j), one 16-byte load each, whole lines per wave.  Rows whose length, pitch or
// address does not allow 16-byte accesses (16-bit output only) take element
// t + T (8 j + i) instead, so that a wave's 2-byte accesses are still contiguous.
#include "dev_common.h"
#include "gemm_common.h"
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

// Largest absolute value as a bit pattern: unsigned order puts infinities above every
// finite value and NaNs above those, so a row with either is seen as such.
__device__ __forceinline__ unsigned abs_bits(float v) { return f_bits(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ unsigned wave_max_u(unsigned v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = max(v, (unsigned)__shfl_xor((int)v, o, 64));
  return v;
}

template <int DT>
__device__ __forceinline__ float add16(float x, float r, unsigned& bits) {
  const unsigned u = cvt_pair<DT>(x + r, 0.0f) & 0xFFFFu;
  bits = u;
  float lo, hi;
  decode2<DT>(u, lo, hi);
  return lo;
}

// QUANT: codes and scales instead of y.  VEC: 16-byte accesses.  T threads a row.
template <int DT, bool QUANT, bool DUAL, bool VEC, int NP>
__global__ __launch_bounds__(1024) void k_rmsnorm(NormArgs a, int T) {
  static_assert(VEC || !QUANT, "codes are written 8 at a time");
  static_assert(QUANT || !DUAL, "the outlier partition is one of codes");
  __shared__ double s_sum[16];
  __shared__ unsigned s_max[16][2];
  __shared__ unsigned s_mask[DUAL ? 1024 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wpr = T >> 6;            // waves per row
  const int rpb = (int)blockDim.x / T;
  const int rib = wave / wpr;
  const int lt = tid - rib * T;

  auto elem = [&](int j, int i) { return VEC ? 8 * (lt + T * j) + i : lt + T * (8 * j + i); };

  float wv[NP][8];
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = min(elem(j, i), a.k - 1);
      wv[j][i] = !a.w ? 1.0f : a.w_f32 ? reinterpret_cast<const float*>(a.w)[e] : load1<DT>(a.w, e);
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
      const int e = elem(j, 0);
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

  for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < a.rows; row0 += (int64_t)gridDim.x * rpb) {
    const int64_t row = row0 + rib;
    const bool row_ok = row < a.rows;
    const int64_t rr = row_ok ? row : a.rows - 1;
    const uint16_t* xr = a.x + rr * a.ldx;
    const uint16_t* sr = a.res ? a.res + rr * a.ldr : nullptr;
    float v[NP][8];
    unsigned hb[NP][8];  // bit patterns of h
    if constexpr (VEC) {
      u4v raw[NP], rad[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int e = elem(j, 0) < a.k ? elem(j, 0) : 0;
        raw[j] = *reinterpret_cast<const u4v*>(xr + e);
        if (sr) rad[j] = *reinterpret_cast<const u4v*>(sr + e);
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          decode2<DT>(raw[j][i], v[j][2 * i], v[j][2 * i + 1]);
          hb[j][2 * i] = raw[j][i] & 0xFFFFu;
          hb[j][2 * i + 1] = raw[j][i] >> 16;
        }
        if (sr) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float lo, hi;
            decode2<DT>(rad[j][i], lo, hi);
            v[j][2 * i] = add16<DT>(v[j][2 * i], lo, hb[j][2 * i]);
            v[j][2 * i + 1] = add16<DT>(v[j][2 * i + 1], hi, hb[j][2 * i + 1]);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = min(elem(j, i), a.k - 1);
          hb[j][i] = xr[e];
          v[j][i] = load1<DT>(xr, e);
          if (sr) v[j][i] = add16<DT>(v[j][i], load1<DT>(sr, e), hb[j][i]);
        }
    }
    // The outlier channels' h, gathered before anyone stores h (h may be x or r itself).
    float ov[2] = {0.0f, 0.0f};
    if constexpr (DUAL) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (oidx[i] >= 0) {
          ov[i] = load1<DT>(xr, oidx[i]);
          unsigned t;
          if (sr) ov[i] = add16<DT>(ov[i], load1<DT>(sr, oidx[i]), t);
          ov[i] = f32_fence(ov[i]);
        }
    }
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (elem(j, i) < a.k) ss += (double)v[j][i] * (double)v[j][i];
    ss = wave_sum_d(ss);
    if (wpr > 1) {
      __syncthreads();
      if (lane == 0) s_sum[wave] = ss;
      __syncthreads();
      ss = 0.0;
      for (int w = 0; w < wpr; ++w) ss += s_sum[rib * wpr + w];
    }
    const float rstd = (float)(1.0 / sqrt(ss / (double)a.k + a.eps));

    if (a.h && row_ok) {
      uint16_t* hr = a.h + row * a.ldh;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        if constexpr (VEC) {
          if (elem(j, 0) < a.k) {
            u4v o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = hb[j][2 * i] | (hb[j][2 * i + 1] << 16);
            *reinterpret_cast<u4v*>(hr + elem(j, 0)) = o;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (elem(j, i) < a.k) hr[elem(j, i)] = (uint16_t)hb[j][i];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = (v[j][i] * rstd) * wv[j][i];

    if constexpr (!QUANT) {
      if (row_ok) {
        uint16_t* yr = a.y + row * a.ldy;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          if constexpr (VEC) {
            if (elem(j, 0) < a.k) {
              u4v o;
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = cvt_pair<DT>(v[j][2 * i], v[j][2 * i + 1]);
              *reinterpret_cast<u4v*>(yr + elem(j, 0)) = o;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (elem(j, i) < a.k) yr[elem(j, i)] = (uint16_t)(cvt_pair<DT>(v[j][i], 0.0f) & 0xFFFFu);
          }
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
      if (!a.sgiven) {
        unsigned m0 = 0u, m1 = 0u;
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (elem(j, 0) < a.k) m0 = max(m0, abs_bits(v[j][i]));
        m0 = wave_max_u(m0);
        if constexpr (DUAL) m1 = wave_max_u(max(abs_bits(ov[0]), abs_bits(ov[1])));
        if (wpr > 1) {
          if (lane == 0) {
            s_max[wave][0] = m0;
            s_max[wave][1] = m1;
          }
          __syncthreads();
          for (int w = 0; w < wpr; ++w) {
            m0 = max(m0, s_max[rib * wpr + w][0]);
            if constexpr (DUAL) m1 = max(m1, s_max[rib * wpr + w][1]);
          }
        }
        float s0, s1 = 0.0f;
        dyn_scale(bits_f(m0), qf, r0, s0);
        if (m0 >= 0x7F800000u) {  // an infinity or NaN in the row: its scale says so
          r0 = 0.0f;
          s0 = bits_f(0x7FC00000u);
        }
        if constexpr (DUAL) {
          dyn_scale(bits_f(m1), qf, r1, s1);
          if (m1 >= 0x7F800000u) {
            r1 = 0.0f;
            s1 = bits_f(0x7FC00000u);
          }
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
          if (elem(j, 0) < a.k) {
            unsigned u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = qbyte(v[j][i], r0, qf);
            *reinterpret_cast<u2v*>(cr + elem(j, 0)) =
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

template <int DT, bool QUANT, bool DUAL, bool VEC>
static void launch_norm_np(const NormArgs& a, int np, int grid, int block, int T, hipStream_t st) {
  switch (np) {
    case 1: hipLaunchKernelGGL((k_rmsnorm<DT, QUANT, DUAL, VEC, 1>), dim3(grid), dim3(block), 0, st, a, T); break;
    case 2: hipLaunchKernelGGL((k_rmsnorm<DT, QUANT, DUAL, VEC, 2>), dim3(grid), dim3(block), 0, st, a, T); break;
    default: hipLaunchKernelGGL((k_rmsnorm<DT, QUANT, DUAL, VEC, 4>), dim3(grid), dim3(block), 0, st, a, T); break;
  }
}

template <int DT>
static void launch_norm_dt(const NormArgs& a, bool quant, bool vec, int np, int grid, int block, int T, hipStream_t st) {
  if (quant) {
    if (a.n_out) launch_norm_np<DT, true, true, true>(a, np, grid, block, T, st);
    else launch_norm_np<DT, true, false, true>(a, np, grid, block, T, st);
  } else {
    if (vec) launch_norm_np<DT, false, false, true>(a, np, grid, block, T, st);
    else launch_norm_np<DT, false, false, false>(a, np, grid, block, T, st);
  }
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
  auto wide = [](const void* q, int64_t ld) { return !q || ((reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ld % 8 == 0); };
  const bool vec = quant || (p.k % 8 == 0 && wide(p.x, p.ldx) && wide(p.res, p.ldr) && wide(p.h, p.ldh) && wide(p.y, p.ldy));
  const int pieces = (int)((p.k + 7) / 8);
  int T = 64;
  while (T < 1024 && T * 4 < pieces) T *= 2;
  const int per = (pieces + T - 1) / T;
  const int np = per <= 1 ? 1 : per <= 2 ? 2 : 4;
  const int block = T < 256 ? 256 : T;
  const int64_t need = (p.rows + block / T - 1) / (block / T);
  const int grid = (int)(need < 16384 ? need : 16384);
  if (p.dtype == DT_BF16) launch_norm_dt<DT_BF16>(a, quant, vec, np, grid, block, T, st);
  else launch_norm_dt<DT_F16>(a, quant, vec, np, grid, block, T, st);
  return hipGetLastError();
}

}  // namespace vq_internal
