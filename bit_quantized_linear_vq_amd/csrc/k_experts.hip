// Matrix products of several experts in one launch for gfx950: the rows of A, sorted by
// expert, meet the weights of their own expert.  Two kinds share the tiling: int8 codes
// times packed 8-bit or 4-bit weight codes with the dequantizing epilogue of the integer
// GEMM (the same arithmetic, so a row's output equals that GEMM's bit for bit), and
// 16-bit rows times 16-bit weights with float32 accumulation.
//
// The rows' distribution is known on the device only: offsets[e] .. offsets[e + 1] are
// expert e's rows.  A launch covers the most tiles that any distribution of the rows can
// have, and a workgroup finds its tile from the offsets (a prefix sum of the experts' tile
// counts, 64 experts per wave step) or ends.
#include <type_traits>

#include "dev_common.h"
#include "gemm_common.h"
#include "vq_internal.h"

namespace vqk {

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
  int vec_store;
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

__device__ __forceinline__ v4i unpack4(u2v w) {
  const unsigned h0 = w.x & 0xF0F0F0F0u, l0 = (w.x << 4) & 0xF0F0F0F0u;
  const unsigned h1 = w.y & 0xF0F0F0F0u, l1 = (w.y << 4) & 0xF0F0F0F0u;
  v4i r;
  r.x = (int)__builtin_amdgcn_perm(h0, l0, 0x05010400u);
  r.y = (int)__builtin_amdgcn_perm(h0, l0, 0x07030602u);
  r.z = (int)__builtin_amdgcn_perm(h1, l1, 0x05010400u);
  r.w = (int)__builtin_amdgcn_perm(h1, l1, 0x07030602u);
  return r;
}

// One wave per 32 x 32 block of outputs, operands straight from memory into registers.
// A step is 32 bytes of an A row: 32 codes or 16 elements.
template <int KIND, int OUT_DT>
__global__ __launch_bounds__(64) void k_experts_block(XArgs g) {
  constexpr bool INT = KIND == X_I8 || KIND == X_I4;
  typedef typename std::conditional<KIND == X_BF16, __bf16, _Float16>::type in_t;
  typedef in_t in8 __attribute__((ext_vector_type(8)));
  RowTile tl;
  if (!find_tile(g, 32, blockIdx.x, tl)) return;
  const int lane = threadIdx.x, rl = lane & 31, kc = lane >> 5;
  const int n0 = blockIdx.y * 32;
  const int row = tl.r0 + rl;
  const bool row_ok = row < tl.r1;
  int ar = row_ok ? row : tl.r0;
  if (g.rows) ar = g.rows[ar];
  const bool a_ok = ar >= 0 && ar < g.m_a;  // an index outside a gives a row of zeros
  ar = a_ok ? ar : 0;
  const uint8_t* pa = g.a + ar * g.lda + 16 * kc;
  const uint8_t* pb = g.b + tl.e * g.b_expert + (int64_t)min(n0 + rl, g.n - 1) * g.ldb;
  const int steps = INT ? g.k / 32 : g.k / 16;
  typedef typename std::conditional<INT, v16i, v16f>::type acc_t;
  acc_t acc = acc_t{};
  for (int s = 0; s < steps; ++s) {
    const v4i fa = *reinterpret_cast<const v4i*>(pa + 32 * s);
    const int c = KIND == X_I4 ? 16 * s + 8 * kc : 32 * s + 16 * kc;  // byte of the weight row
    const uint8_t* q = pb + (int64_t)(c >> 6) * g.b_piece + (c & 63);
    if constexpr (KIND == X_I4) {
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(unpack4(*reinterpret_cast<const u2v*>(q)), fa, acc, 0, 0, 0);
    } else {
      const v4i fb = *reinterpret_cast<const v4i*>(q);
      if constexpr (KIND == X_I8) acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb, fa, acc, 0, 0, 0);
      else if constexpr (KIND == X_F16)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(in8, fb), __builtin_bit_cast(in8, fa), acc, 0, 0, 0);
      else
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(in8, fb), __builtin_bit_cast(in8, fa), acc, 0, 0, 0);
    }
  }
  if (!row_ok) return;
  const float sa = INT ? g.sa[ar] : 1.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int n = n0 + 8 * q + 4 * kc + r;
      if (n >= g.n) continue;
      float v;
      if constexpr (INT) {
        int a0 = acc[4 * q + r];
        if constexpr (KIND == X_I4) a0 >>= 4;
        v = (float)a0 * (sa * g.sb[(int64_t)tl.e * g.n + n]);
      } else {
        v = acc[4 * q + r];
      }
      if (!a_ok) v = 0.0f;
      const int64_t o = (int64_t)row * g.ldy + n;
      if constexpr (OUT_DT == DT_F32) reinterpret_cast<float*>(g.y)[o] = v;
      else reinterpret_cast<uint16_t*>(g.y)[o] = (uint16_t)(cvt_pair<OUT_DT>(v, 0.0f) & 0xFFFFu);
    }
}

template <int KIND>
static hipError_t launch_kind(const XArgs& a, int out_dt, hipStream_t st) {
  const int64_t tiles = a.t / 32 + (a.experts < a.t ? a.experts : a.t);
  const dim3 grid((unsigned)tiles, (unsigned)((a.n + 31) / 32));
  switch (out_dt) {
    case DT_F16: hipLaunchKernelGGL((k_experts_block<KIND, DT_F16>), grid, dim3(64), 0, st, a); break;
    case DT_BF16: hipLaunchKernelGGL((k_experts_block<KIND, DT_BF16>), grid, dim3(64), 0, st, a); break;
    default: hipLaunchKernelGGL((k_experts_block<KIND, DT_F32>), grid, dim3(64), 0, st, a); break;
  }
  return hipGetLastError();
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
  const int64_t esize = p.out_dt == DT_F32 ? 4 : 2;
  a.vec_store = ((reinterpret_cast<uintptr_t>(p.y) & 15u) == 0 && (p.ldy * esize) % 16 == 0) ? 1 : 0;
  switch (p.kind) {
    case X_I8: return launch_kind<X_I8>(a, p.out_dt, st);
    case X_I4: return launch_kind<X_I4>(a, p.out_dt, st);
    case X_F16: return launch_kind<X_F16>(a, p.out_dt, st);
    default: return launch_kind<X_BF16>(a, p.out_dt, st);
  }
}

}  // namespace vq_internal
