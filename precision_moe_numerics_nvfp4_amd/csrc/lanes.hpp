// Exchanges between the lanes of a wavefront by register operands, without LDS.
#pragma once

#include "codecs.hpp"

namespace nvfp4moe {

// The value of the lane across in a group of 2, 4, 8, 16 (each step reaches the
// half of its group that the earlier ones did not): DPP operands, no LDS.
template <int STEP>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  constexpr int ctrl = STEP == 0 ? 0xB1 /* quad_perm 1,0,3,2 */
                       : STEP == 1 ? 0x4E /* quad_perm 2,3,0,1 */
                       : STEP == 2 ? 0x141 /* row_half_mirror */ : 0x140 /* row_mirror */;
  return __builtin_amdgcn_update_dpp(v, v, ctrl, 0xF, 0xF, true);
}
template <int STEP>
__device__ __forceinline__ float across(float v) { return u2f(across<STEP>(f2u(v))); }
template <int STEP>
__device__ __forceinline__ int across(int v) { return (int)across<STEP>((uint32_t)v); }
template <int STEP>
__device__ __forceinline__ double across(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint64_t r = ((uint64_t)across<STEP>((uint32_t)(u >> 32)) << 32) | across<STEP>((uint32_t)u);
  return __longlong_as_double((int64_t)r);
}

// A value joined over the four rows of 16 lanes, lane by lane: the two halves of
// each pair of rows, then of the wavefront, meet in the results of a row swap.
template <class T, class Op>
__device__ __forceinline__ T join_rows(T v, Op op) {
  static_assert(sizeof(T) == 4);
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  v = op(__builtin_bit_cast(T, r0), __builtin_bit_cast(T, r1));
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  const uint32_t q0 = q[0], q1 = q[1];
  return op(__builtin_bit_cast(T, q0), __builtin_bit_cast(T, q1));
}

// Orders the LDS accesses of one wavefront's lanes before and after it (the
// hardware runs them in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace nvfp4moe
