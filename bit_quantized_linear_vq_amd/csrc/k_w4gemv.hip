// 4-bit weights with a scale for each group of 32, 64 or 128 input channels, and their
// product with a few 16-bit rows: the linear layer's form for single tokens, where the
// weights' bytes are all that counts and activations stay at 16 bits.
//
//   s[j,g] = RNE16(fl32(max|w| / 7)),  c[j,k] = clamp(rne(fl32(w * fl32(1 / s))), -7, 7)
//   y[i,j] = sum_g s[j,g] * sum_{k in g} c[j,k] x[i,k]      (float32)
#include <algorithm>
#include <type_traits>

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
    // An infinity or NaN makes its group's maximum infinite (fmaxf alone would pass a NaN by).
    float m = 0.0f, z = 0.0f;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      m = fmaxf(m, fabsf(v[t]));
      z += v[t] * 0.0f;
    }
    if (!(z == 0.0f)) m = bits_f(0x7F800000u);
    if (!ok) m = 0.0f;
#pragma unroll
    for (int o = LPG / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    const bool bad = !(m < bits_f(0x7F800000u));
    const unsigned s16 = bad ? (DT == DT_BF16 ? 0x7FC0u : 0x7E00u) : cvt_pair<DT>(m / 7.0f, 0.0f) & 0xFFFFu;
    float s, unused;
    decode2<DT>(s16, s, unused);
    float r = 1.0f / s;
    if (!(s > 0.0f) || __builtin_isinf(r)) r = 0.0f;
    if (ok) {
      unsigned u[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) u[t] = qbyte(bad ? 0.0f : v[t], r, 7.0f);
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
  int m, n, k, group, out_dt;
  int tile;  // rows of x per workgroup, 16 MB at most
};

// ---------------------------------------------------------------------------------------
// The product on the 16 x 16 x 32 matrix instruction: 16 rows of x against 16 output
// channels, so that up to 16 rows cost what one does.
//
// Codes become exact 16-bit floats before they meet x (see widen).  Leaving them at c + 24, which
// costs one and-or for two, and taking 24 sum x off the accumulators was faster with
// bfloat16 rows (below), but rounded a loud channel of x at 24 to 31 times its size even where its
// code is 0 (error 0.1% of the outputs at 1e5 among unit values) and lost finite rows above 1e37.
//
// Layout: a lane loads 16 bytes of a weight row, 32 codes, the 64 lanes 64 bytes of 16
// rows.  A matrix instruction wants 32 consecutive channels spread over the lanes' four
// groups of 16, 8 each, so the 4 x 4 dwords of the four lanes of a row are transposed by
// two swaps between half-waves and two between rows of 16 lanes.  Instruction j of a 64-byte
// piece then covers channels 32 j .. 32 j + 31, never two groups, and dword pairs (t, t + 4)
// of x meet the codes' pairs.
//
// A lane's accumulators hold one output channel (lane mod 16) and rows 4 (lane div 16) + i, so
// a group's scale is one value per lane: y += s * acc.
//
// A workgroup's waves (four, eight, or KS where that is more) take KS parts of K times blocks of 16
// channels.  x goes through LDS in chunks of 4 pieces (512 channels) of every part, its pairs
// put in order once per workgroup (rows 1040 bytes apart: 16 rows then read 16 bytes each
// without a bank conflict); the weights come straight to registers, a chunk ahead (two ahead
// was even or slower: it costs registers, and with them waves).  The parts are joined through
// LDS in a fixed order.
//
// Measured, with the launch, bfloat16 / fp16 rows (in brackets with codes left at c + 24): 4096 -> 12288,
// one row, groups of 64, 10.4 / 9.6 us (9.5 / 9.6); 8192 -> 28672, one row, groups of 128, 34.4 / 31.1 us = 3.5
// / 3.9 TB/s (30.0 / 29.9); 8192 -> 28671, seven rows, groups of 32, 42.9 / 41.1 us = 3.1 / 3.2 TB/s (40.3 /
// 40.4); 32 rows, groups of 128, 8192 -> 8192 24.2 / 22.2 us (22.1 / 22.3), 8192 -> 28672 53.0 / 49.9 (51.9 /
// 51.3).  For every 512 codes a wave has 35 / 25 vector instructions with groups of 32, 29 / 20 with 128: the
// vector units are busy 55% / 40% of the seven rows' time, 53% / 39% of the one row's, and on average 2.2
// waves of a possible 4 are there, as the last workgroups end.
// Two blocks of channels a wave (x read from LDS once for both) was slower nearly everywhere
// (8192 -> 28672 32.0 against 30.2 us, codes at c + 24): half the waves.
constexpr int GV_SETS = 2;
constexpr int GV_CHUNK = 4;                         // pieces
constexpr int GV_ROW = GV_CHUNK * 256 + 16;         // bytes of a row of a chunk of x in LDS
constexpr int GV_ROWS = 32;                         // rows times parts at most

template <int DT, int GROUP, int KS, int MB, int XL, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(KS == 16 ? 4 : 3))) void k_w4gemv(GemvArgs g) {
  typedef typename std::conditional<DT == DT_BF16, __bf16, _Float16>::type in_t;
  typedef in_t in8 __attribute__((ext_vector_type(8)));
  constexpr int GPP = 128 / GROUP;     // groups of a piece
  constexpr int GPC = GPP * GV_CHUNK;  // and of a chunk
  extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];  // [2][part][row][GV_ROW]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rl = lane & 15, kq = lane >> 4;
  const int kw = wave % KS, nw = wave / KS;
  const int n0 = ((int)blockIdx.x * (WAVES / KS) + nw) * 16, m0 = blockIdx.y * g.tile;
  const int rows = min(g.tile, g.m - m0);
  const int pieces = (g.k + 127) / 128;
  const int p0 = pieces * kw / KS, p1 = pieces * (kw + 1) / KS;
  const int chunks = ((pieces + KS - 1) / KS + GV_CHUNK - 1) / GV_CHUNK;  // of the longest part
  const int groups = g.k / GROUP;
  const int64_t jn = min(n0 + rl, g.n - 1);
  const uint8_t* pw = g.codes + jn * (g.k / 2);
  const uint16_t* ps = g.scales + jn * groups;

  v4i w[GV_SETS][GV_CHUNK];
  unsigned sc[GV_SETS][GPC / 2];  // two scales each
  auto load_w = [&](int set, int c) __attribute__((always_inline)) {
    const int q0 = p0 + GV_CHUNK * c;
    if (q0 >= p1) return;
#pragma unroll
    for (int u = 0; u < GV_CHUNK; ++u) {
      // Past the part's end or the row's last group: the row's first bytes, not used.
      const int at = q0 + u < p1 && 128 * (q0 + u) + 32 * kq < g.k ? 64 * (q0 + u) + 16 * kq : 0;
      w[set][u] = *reinterpret_cast<const v4i*>(pw + at);
    }
    const int g0 = q0 * GPP;
    if (g0 + GPC <= groups) {
      typedef unsigned vec __attribute__((ext_vector_type(GPC / 2 <= 4 ? GPC / 2 : 4)));
      typedef vec vec_any __attribute__((aligned(2)));
#pragma unroll
      for (int t = 0; t < GPC; t += 8) {
        const vec v = *reinterpret_cast<const vec_any*>(ps + g0 + t);
#pragma unroll
        for (int e = 0; e < (GPC < 8 ? GPC : 8) / 2; ++e) sc[set][t / 2 + e] = v[e];
      }
    } else {
#pragma unroll
      for (int t = 0; t < GPC; t += 2)
        sc[set][t / 2] = ps[min(g0 + t, groups - 1)] | ((unsigned)ps[min(g0 + t + 1, groups - 1)] << 16);
    }
  };
  v4i xr[XL];
  auto load_x = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < XL; ++t) {
      const int rp = wave + WAVES * t, part = rp % KS, row = rp / KS;
      if (row >= rows) break;
      const int q0 = pieces * part / KS + GV_CHUNK * c, q1 = pieces * (part + 1) / KS;
      const int at = 128 * q0 + 8 * lane;
      xr[t] = at < min(g.k, 128 * q1) ? *reinterpret_cast<const v4i*>(g.x + (m0 + row) * g.ldx + at) : v4i{};
    }
  };
  auto store_x = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < XL; ++t) {
      const int rp = wave + WAVES * t, part = rp % KS, row = rp / KS;
      if (row >= rows) break;
      const v4i v = xr[t];
      // dword pairs (e, e + 4)
      const v4i o = {(int)__builtin_amdgcn_perm((unsigned)v.z, (unsigned)v.x, 0x05040100u),
                     (int)__builtin_amdgcn_perm((unsigned)v.z, (unsigned)v.x, 0x07060302u),
                     (int)__builtin_amdgcn_perm((unsigned)v.w, (unsigned)v.y, 0x05040100u),
                     (int)__builtin_amdgcn_perm((unsigned)v.w, (unsigned)v.y, 0x07060302u)};
      *reinterpret_cast<v4i*>(s_x + ((buf * KS + part) * rows + row) * GV_ROW + 16 * lane) = o;
    }
  };
  auto mma = [&](v4i a, v4i b, v4f c) {
    if constexpr (DT == DT_BF16)
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(in8, a), __builtin_bit_cast(in8, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(in8, a), __builtin_bit_cast(in8, b), c, 0, 0, 0);
  };
  // Eight codes of a dword as exact 16-bit floats, pairs (t, t + 4); u = c + 8 is one exclusive or for
  // all.  fp16: u in the top four mantissa bits of 16.0, two of them per shift and and-or, then 24 off both
  // in one packed subtraction.  bfloat16 has no packed arithmetic: u stays where it lies in the dword, as the
  // mantissa bits of a float32 whose last of them counts one (2^23 for bits 0-3, 2^19 for bits 4-7, ...), one
  // and-or and one exact subtraction, and the upper halves of two such floats make a pair.  The
  // constants are kept in registers: and-or takes no literals.
  unsigned mask[4], one[4];
  if constexpr (DT == DT_BF16) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      mask[t] = 0xFu << (4 * t);
      one[t] = (unsigned)(127 + 23 - 4 * t) << 23;
      asm("" : "+v"(mask[t]), "+s"(one[t]));
    }
  } else {
    mask[0] = 0x03C003C0u;
    one[0] = 0x4C004C00u;
    asm("" : "+v"(mask[0]), "+s"(one[0]));
  }
  auto widen = [&](unsigned c) {
    const unsigned u = c ^ 0x88888888u;
    v4i o;
    if constexpr (DT == DT_BF16) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float excess = (float)(1 << (23 - 4 * t)) + 8.0f;
        const float lo = bits_f((u & mask[t]) | one[t]) - excess;
        const float hi = bits_f(((u >> 16) & mask[t]) | one[t]) - excess;
        o[t] = (int)__builtin_amdgcn_perm(f_bits(hi), f_bits(lo), 0x07060302u);
      }
    } else {
      typedef _Float16 h2 __attribute__((ext_vector_type(2)));
      const unsigned at[4] = {u << 6, u << 2, u >> 2, u >> 6};
#pragma unroll
      for (int t = 0; t < 4; ++t)
        o[t] = __builtin_bit_cast(int, __builtin_bit_cast(h2, (at[t] & mask[0]) | one[0]) - h2{(_Float16)24.0f, (_Float16)24.0f});
    }
    return o;
  };

  v4f y[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) y[i] = v4f{};
  // whole: every piece of the chunk is there in full (no branch between the pieces).
  auto compute = [&](auto whole, int set, int buf, int c) __attribute__((always_inline)) {
    const uint8_t* xb[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
      xb[i] = s_x + ((buf * KS + kw) * rows + min(16 * i + rl, rows - 1)) * GV_ROW + 16 * kq;
#pragma unroll
    for (int u = 0; u < GV_CHUNK; ++u) {
      const int q = p0 + GV_CHUNK * c + u;
      if (!decltype(whole)::value && q >= p1) break;
      const v4i t = w[set][u];
      const auto r02 = __builtin_amdgcn_permlane32_swap((unsigned)t.x, (unsigned)t.z, false, false);
      const auto r13 = __builtin_amdgcn_permlane32_swap((unsigned)t.y, (unsigned)t.w, false, false);
      const auto e01 = __builtin_amdgcn_permlane16_swap(r02[0], r13[0], false, false);
      const auto e23 = __builtin_amdgcn_permlane16_swap(r02[1], r13[1], false, false);
      const unsigned wt[4] = {e01[0], e01[1], e23[0], e23[1]};
#pragma unroll
      for (int j0 = 0; j0 < 4; j0 += GROUP / 32) {
        if (!decltype(whole)::value && 128 * q + 32 * j0 >= g.k) break;
        v4i xf[GROUP / 32][MB];
        v4f acc[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          acc[i] = v4f{};
#pragma unroll
          for (int j = 0; j < GROUP / 32; ++j) xf[j][i] = *reinterpret_cast<const v4i*>(xb[i] + 256 * u + 64 * (j0 + j));
        }
        float s0, s1;
        const int si = u * GPP + j0 / (GROUP / 32);
        decode2<DT>(sc[set][si / 2], s0, s1);
        const float s = si & 1 ? s1 : s0;
#pragma unroll
        for (int j = 0; j < GROUP / 32; ++j) {
          const v4i wf = widen(wt[j0 + j]);
#pragma unroll
          for (int i = 0; i < MB; ++i) acc[i] = mma(xf[j][i], wf, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) y[i][r] = __builtin_fmaf(s, acc[i][r], y[i][r]);
      }
    }
  };
  load_x(0);
#pragma unroll
  for (int i = 0; i < GV_SETS - 1; ++i) load_w(i, i);
  store_x(0);
  __syncthreads();
  for (int c0 = 0; c0 < chunks; c0 += GV_SETS) {
#pragma unroll
    for (int i = 0; i < GV_SETS; ++i) {
      const int c = c0 + i;
      if (c < chunks) {
        if (c + 1 < chunks) load_x(c + 1);
        load_w((i + GV_SETS - 1) % GV_SETS, c + GV_SETS - 1);
        const int qe = p0 + GV_CHUNK * (c + 1);
        if (qe <= p1 && 128 * qe <= g.k) compute(std::true_type{}, i, c & 1, c);
        else compute(std::false_type{}, i, c & 1, c);
        if (c + 1 < chunks) store_x((c + 1) & 1);
        __syncthreads();
      }
    }
  }
  if constexpr (KS > 1) {
    v4f* part = reinterpret_cast<v4f*>(s_x);  // [wave][MB][64]
#pragma unroll
    for (int i = 0; i < MB; ++i) part[(wave * MB + i) * 64 + lane] = y[i];
    __syncthreads();
    if (kw) return;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int q = 1; q < KS; ++q) y[i] += part[((wave + q) * MB + i) * 64 + lane];
  }
  const int n = n0 + rl;
  if (n >= g.n) return;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = m0 + 16 * i + 4 * kq + r;
      if (m >= m0 + rows) continue;
      const int64_t o = m * g.ldy + n;
      if (g.out_dt == DT_F32) reinterpret_cast<float*>(g.y)[o] = y[i][r];
      else reinterpret_cast<uint16_t*>(g.y)[o] = (uint16_t)((g.out_dt == DT_BF16 ? cvt_pair<DT_BF16>(y[i][r], 0.0f) : cvt_pair<DT_F16>(y[i][r], 0.0f)) & 0xFFFFu);
    }
}

constexpr size_t GV_LDS = 160 * 1024;  // of a compute unit
static size_t gv_shared(int ks, int mb, int rows, int waves) {
  return std::max((size_t)2 * ks * rows * GV_ROW, (size_t)waves * mb * 64 * 16);  // x, or the parts' joining
}

template <int DT, int GROUP, int KS, int MB, int WAVES>
static void launch_gemv_waves(const GemvArgs& a, hipStream_t st) {
  constexpr int COLS = 16 * WAVES / KS;
  const int rows = a.tile;
  const size_t shm = gv_shared(KS, MB, rows, WAVES);
  const dim3 grid((unsigned)((a.n + COLS - 1) / COLS), (unsigned)((a.m + rows - 1) / rows));
  const int loads = (rows * KS + WAVES - 1) / WAVES;  // of x, per thread and chunk
#define VQ_GEMV_XL(X) hipLaunchKernelGGL((k_w4gemv<DT, GROUP, KS, MB, X, WAVES>), grid, dim3(64 * WAVES), shm, st, a)
  if constexpr (MB == 2) {
    VQ_GEMV_XL(8);
  } else if constexpr (KS == 16) {
    if (loads <= 1) VQ_GEMV_XL(1);
    else VQ_GEMV_XL(2);
  } else if constexpr (WAVES == 8 && KS < 8) {
    VQ_GEMV_XL(4);
  } else {
    if (loads <= 1) VQ_GEMV_XL(1);
    else if (loads <= 2) VQ_GEMV_XL(2);
    else if constexpr (KS == 8) VQ_GEMV_XL(4);
    else if (loads <= 4) VQ_GEMV_XL(4);
    else VQ_GEMV_XL(8);
  }
#undef VQ_GEMV_XL
}

template <int DT, int GROUP, int KS>
static void launch_gemv_part(const GemvArgs& a, hipStream_t st) {
  if constexpr (KS > 4) {
    launch_gemv_waves<DT, GROUP, KS, 1, KS>(a, st);
  } else {
    // Many rows of x leave LDS (above 16 rows and parts also registers) for fewer than the four
    // workgroups of four waves that a compute unit can hold: eight waves then share the same x,
    // unless all workgroups fit at once.  8192 -> n, bfloat16, groups of 128, 4 / 8 waves, us: 16 rows, n =
    // 16384 24.6 / 27.7, 20480 44.0 / 38.6, 28672 52.5 / 41.0; 8 rows, n = 8192 14.7 / 15.6, 12288
    // 24.3 / 21.2; groups of 32, 9 rows, 28672 54.2 / 43.8, 7 rows 42.9 / 43.1 but 24576 35.9 / 42.7.
    const int fit = std::min((int)(GV_LDS / gv_shared(KS, 1, a.tile, 4)), a.tile * KS > 16 ? 3 : 4);
    const int64_t groups = ((int64_t)a.n * KS + 63) / 64 * ((a.m + a.tile - 1) / a.tile);
    if (fit < 4 && groups > (int64_t)fit * vq_internal::persistent_blocks()) launch_gemv_waves<DT, GROUP, KS, 1, 8>(a, st);
    else launch_gemv_waves<DT, GROUP, KS, 1, 4>(a, st);
  }
}

template <int DT, int GROUP>
static void launch_gemv_group(GemvArgs a, hipStream_t st) {
  // Parts of K: waves enough for the whole card, at least two.  One bfloat16 row, us with 2 / 4 / 8 / 16
  // parts: 16384 -> 2048 30.1 / 17.1 / 13.2 / 11.7; 8192 -> 8192 17.0 / 12.0 / 12.7 / 16.5; 4096 ->
  // 14336 11.2 / 11.6 / 11.3 / 20.2; 8192 -> 28672 34.9 / 32.6 / 35.4 / 50.2 (fp16 31.0 / 29.5 / 33.9 / 46.2:
  // the rule's two give up 5 to 7% there); seven rows, groups of 32, 8192 -> 28671 42.9 / 47.3.  Many rows of
  // x leave room in LDS for fewer parts.
  const int64_t blocks = ((int64_t)a.n + 15) / 16;
  int ks = 2;
  while (ks < 16 && ks * blocks < 1600) ks *= 2;
  a.tile = a.m;
  if (a.m > 4) {
    // Fewer rows a workgroup leave room for more parts, as long as all waves are there at once
    // (16 a compute unit; the weights' further readings come from the caches).  Us with tiles of 32 / 16 /
    // 8 / 4 rows and 1 / 2 / 4 / 8 parts, bfloat16: 32 rows, 16384 -> 2048 83.9 / 40.7 / 24.6 / 38.1, 8192 ->
    // 8192 43.6 / 25.5 / 38.8 / 71.9, 8192 -> 28672 52.9 / 73.0 / 129 / 242; 16 rows, 8192 -> 512 - / 19.0 / 11.0 /
    // 8.2, 4096 - / 21.7 / 14.8 / 22.5, 4096 -> 12288 - / 14.2 / 17.7 / 34.8.
    for (int tile = 4; tile <= 16; tile *= 2) {
      const int parts = GV_ROWS / tile;
      const int64_t tiles = (a.m + tile - 1) / tile;
      if (parts > ks || parts * blocks * tiles > 16 * (int64_t)vq_internal::persistent_blocks()) continue;
      ks = parts;
      a.tile = (int)((a.m + tiles - 1) / tiles);
      break;
    }
  }
  if (a.tile > 16) {
    a.tile = std::min(a.m, 32);
    launch_gemv_waves<DT, GROUP, 1, 2, 4>(a, st);
    return;
  }
  while (a.tile * ks > GV_ROWS) ks /= 2;
  if (ks == 16) launch_gemv_part<DT, GROUP, 16>(a, st);
  else if (ks == 8) launch_gemv_part<DT, GROUP, 8>(a, st);
  else if (ks == 4) launch_gemv_part<DT, GROUP, 4>(a, st);
  else launch_gemv_part<DT, GROUP, 2>(a, st);
}

template <int DT>
static void launch_gemv_dt(const GemvArgs& a, hipStream_t st) {
  if (a.group == 32) launch_gemv_group<DT, 32>(a, st);
  else if (a.group == 64) launch_gemv_group<DT, 64>(a, st);
  else launch_gemv_group<DT, 128>(a, st);
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
  a.out_dt = p.out_dt;
  if (p.in_dt == DT_BF16) launch_gemv_dt<DT_BF16>(a, st);
  else launch_gemv_dt<DT_F16>(a, st);
  return hipGetLastError();
}

}  // namespace vq_internal
