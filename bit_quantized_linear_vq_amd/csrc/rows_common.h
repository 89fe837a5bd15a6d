// Pieces shared by the row kernels (norms, combining): rows of 16-bit elements in pieces of eight at
// any element's address, and wave-wide sums in float64.
#pragma once

#include "dev_common.h"

namespace vqk {

typedef u4v u4v_el __attribute__((aligned(2)));
typedef v4f v4f_el __attribute__((aligned(4)));

// Wave-wide sum in float64: four steps of register moves inside the rows of 16 lanes, then the
// four rows from scalar registers.
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ double lane_d(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ double wave_sum_dpp(double v) {
  v += dpp_d<0xB1>(v);   // quad_perm [1,0,3,2]
  v += dpp_d<0x4E>(v);   // quad_perm [2,3,0,1]
  v += dpp_d<0x141>(v);  // row_half_mirror
  v += dpp_d<0x140>(v);  // row_mirror
  return (lane_d(v, 0) + lane_d(v, 16)) + (lane_d(v, 32) + lane_d(v, 48));
}

// Eight elements at any element's address; TINY: the row has only cnt < 8; NT: past the cache.
template <bool TINY, bool NT>
__device__ __forceinline__ u4v load8(const uint16_t* p, int cnt) {
  if constexpr (!TINY && NT) return __builtin_nontemporal_load(reinterpret_cast<const u4v_el*>(p));
  if constexpr (!TINY) return *reinterpret_cast<const u4v_el*>(p);
  u4v v = {0u, 0u, 0u, 0u};
  for (int i = 0; i < 8; ++i)
    if (i < cnt) v[i >> 1] |= (unsigned)p[i] << (16 * (i & 1));
  return v;
}
template <bool TINY, bool NT>
__device__ __forceinline__ void store8(uint16_t* p, const u4v& v, int cnt) {
  if constexpr (!TINY && NT) {
    __builtin_nontemporal_store(v, reinterpret_cast<u4v_el*>(p));
  } else if constexpr (!TINY) {
    *reinterpret_cast<u4v_el*>(p) = v;
  } else {
    for (int i = 0; i < 8; ++i)
      if (i < cnt) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
  }
}

// How K ends: a multiple of 8; a last piece that starts early enough to end with the row, its
// first elements counted by their own piece; or fewer than 8 elements in all.
enum : int { END_WHOLE = 0, END_OVERLAP = 1, END_TINY = 2 };

}  // namespace vqk
