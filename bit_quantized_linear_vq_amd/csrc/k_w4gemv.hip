// 4-bit weights with a scale for each group of 32, 64 or 128 input channels, and their
// product with a few 16-bit rows: the linear layer's form for single tokens, where the
// weights' bytes are all that counts and activations stay at 16 bits.
//
//   s[j,g] = RNE16(fl32(max|w| / 7)),  c[j,k] = clamp(rne(fl32(w * fl32(1 / s))), -7, 7)
//   y[i,j] = sum_g s[j,g] * sum_{k in g} c[j,k] x[i,k]      (float32)
#include "dev_common.h"
#include "gemm_common.h"
#include "vq_internal.h"

namespace vqk {

// One lane quantizes 8 weights; LPG lanes share a group.
template <int DT, int LPG>
__global__ __launch_bounds__(256) void k_pack_group(const uint16_t* w, int64_t ldw, int64_t n, int k, uint8_t* codes,
                                                    uint16_t* scales) {
  const int ppr = k / 8;
  const int64_t pieces = n * ppr;
  // whole waves take part in the exchange: every lane of a wave stays in the loop
  for (int64_t i0 = (int64_t)blockIdx.x * 256; i0 < pieces; i0 += (int64_t)gridDim.x * 256) {
    const int64_t i = i0 + threadIdx.x;
    const bool ok = i < pieces;
    const int64_t ii = ok ? i : pieces - 1;
    const int64_t row = ii / ppr;
    const int p = (int)(ii - row * ppr);
    const u4v raw = *reinterpret_cast<const u4v*>(w + row * ldw + 8 * p);
    float v[8];
#pragma unroll
    for (int t = 0; t < 4; ++t) decode2<DT>(raw[t], v[2 * t], v[2 * t + 1]);
    float m = 0.0f;
#pragma unroll
    for (int t = 0; t < 8; ++t) m = fmaxf(m, fabsf(v[t]));
    if (!ok) m = 0.0f;
#pragma unroll
    for (int o = LPG / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    const unsigned s16 = cvt_pair<DT>(m / 7.0f, 0.0f) & 0xFFFFu;
    float s, unused;
    decode2<DT>(s16, s, unused);
    float r = 1.0f / s;
    if (!(s > 0.0f) || __builtin_isinf(r)) r = 0.0f;
    if (ok) {
      unsigned u[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) u[t] = qbyte(v[t], r, 7.0f);
      *reinterpret_cast<unsigned*>(codes + row * (k / 2) + 4 * p) = pack8_nibbles(u);
      if ((p & (LPG - 1)) == 0) scales[row * (ppr / LPG) + p / LPG] = (uint16_t)s16;
    }
  }
}

struct GemvArgs {
  const uint16_t* x;
  const uint8_t* codes;
  const uint16_t* scales;
  void* y;
  int64_t ldx, ldy;
  int m, n, k, group;
};

// One wave per output channel and row.
template <int DT, int OUT_DT>
__global__ __launch_bounds__(256) void k_w4gemv(GemvArgs g) {
  const int lane = threadIdx.x & 63;
  const int j = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (j >= g.n) return;
  const int words = g.k / 8, wpg = g.group / 8;
  for (int i = blockIdx.y; i < g.m; i += gridDim.y) {
    float acc = 0.0f;
    for (int q = lane; q < words; q += 64) {
      const unsigned c = *reinterpret_cast<const unsigned*>(g.codes + (int64_t)j * (g.k / 2) + 4 * q);
      const float s = load1<DT>(g.scales, (int64_t)j * (words / wpg) + q / wpg);
      float part = 0.0f;
#pragma unroll
      for (int t = 0; t < 8; ++t)
        part += (float)((int)(c << (28 - 4 * t)) >> 28) * load1<DT>(g.x, i * g.ldx + 8 * q + t);
      acc += s * part;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) acc += __shfl_xor(acc, o, 64);
    if (lane == 0) {
      if constexpr (OUT_DT == DT_F32) {
        reinterpret_cast<float*>(g.y)[i * g.ldy + j] = acc;
      } else {
        reinterpret_cast<uint16_t*>(g.y)[i * g.ldy + j] = (uint16_t)(cvt_pair<OUT_DT>(acc, 0.0f) & 0xFFFFu);
      }
    }
  }
}

}  // namespace vqk

namespace vq_internal {

using namespace vqk;

hipError_t launch_pack_group(const void* w, int dtype, int64_t n, int64_t k, int64_t ldw, int group, uint8_t* codes,
                             void* scales, hipStream_t st) {
  const int64_t pieces = n * (k / 8);
  const int64_t need = (pieces + 255) / 256;
  const int grid = (int)(need < 65536 ? need : 65536);
  const uint16_t* wp = reinterpret_cast<const uint16_t*>(w);
  uint16_t* sp = reinterpret_cast<uint16_t*>(scales);
#define VQ_PACKG(D, L) hipLaunchKernelGGL((k_pack_group<D, L>), dim3(grid), dim3(256), 0, st, wp, ldw, n, (int)k, codes, sp)
  if (dtype == DT_BF16) {
    if (group == 32) VQ_PACKG(DT_BF16, 4);
    else if (group == 64) VQ_PACKG(DT_BF16, 8);
    else VQ_PACKG(DT_BF16, 16);
  } else {
    if (group == 32) VQ_PACKG(DT_F16, 4);
    else if (group == 64) VQ_PACKG(DT_F16, 8);
    else VQ_PACKG(DT_F16, 16);
  }
#undef VQ_PACKG
  return hipGetLastError();
}

hipError_t launch_w4gemv(const W4GemvParams& p, hipStream_t st) {
  GemvArgs a{};
  a.x = reinterpret_cast<const uint16_t*>(p.x);
  a.codes = p.codes;
  a.scales = reinterpret_cast<const uint16_t*>(p.scales);
  a.y = p.y;
  a.ldx = p.ldx;
  a.ldy = p.ldy;
  a.m = (int)p.m;
  a.n = (int)p.n;
  a.k = (int)p.k;
  a.group = p.group;
  const dim3 grid((unsigned)((p.n + 3) / 4), (unsigned)(p.m < 1024 ? p.m : 1024));
#define VQ_GEMV(I, O) hipLaunchKernelGGL((k_w4gemv<I, O>), grid, dim3(256), 0, st, a)
  if (p.in_dt == DT_BF16) {
    switch (p.out_dt) {
      case DT_F16: VQ_GEMV(DT_BF16, DT_F16); break;
      case DT_BF16: VQ_GEMV(DT_BF16, DT_BF16); break;
      default: VQ_GEMV(DT_BF16, DT_F32); break;
    }
  } else {
    switch (p.out_dt) {
      case DT_F16: VQ_GEMV(DT_F16, DT_F16); break;
      case DT_BF16: VQ_GEMV(DT_F16, DT_BF16); break;
      default: VQ_GEMV(DT_F16, DT_F32); break;
    }
  }
#undef VQ_GEMV
  return hipGetLastError();
}

}  // namespace vq_internal
