// Reductions across the lanes of a wavefront.
#pragma once

#include <hip/hip_runtime.h>

namespace osc {
namespace {

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// max of a value over the lanes that differ in bit 5, and in bits 4 and 5: the swap instructions
// exchange half-wavefronts (16-lane rows) of two registers, so of two copies of v they leave each
// lane its own and its partner's.  (The results are read as integers first: a bit cast straight from a
// vector's element reads element 0 whichever is named.)
__device__ __forceinline__ float max_halves(float v) {
  const unsigned a = __builtin_bit_cast(unsigned, v);
  const auto x = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const unsigned x0 = x[0], x1 = x[1];
  return fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1));
}
__device__ __forceinline__ float max_groups(float v) {
  const unsigned a = __builtin_bit_cast(unsigned, v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const unsigned x0 = x[0], x1 = x[1];
  return max_halves(fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1)));
}

// The same and the sum over all lanes.  A row of 16 lanes first: neighbours, pairs, then the two mirrors.
template <int CTRL>
__device__ __forceinline__ float lane_swap(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float max_wave(float v) {
  v = fmaxf(v, lane_swap<0xB1>(v));
  v = fmaxf(v, lane_swap<0x4E>(v));
  v = fmaxf(v, lane_swap<0x141>(v));
  v = fmaxf(v, lane_swap<0x140>(v));
  return max_groups(v);
}
__device__ __forceinline__ float sum_wave(float v) {
  v += lane_swap<0xB1>(v);
  v += lane_swap<0x4E>(v);
  v += lane_swap<0x141>(v);
  v += lane_swap<0x140>(v);
  const unsigned a = __builtin_bit_cast(unsigned, v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const unsigned x0 = x[0], x1 = x[1];
  const unsigned b = __builtin_bit_cast(unsigned, __builtin_bit_cast(float, x0) + __builtin_bit_cast(float, x1));
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const unsigned y0 = y[0], y1 = y[1];
  return __builtin_bit_cast(float, y0) + __builtin_bit_cast(float, y1);
}

}  // namespace
}  // namespace osc
