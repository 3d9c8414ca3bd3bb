// Reductions over the lanes of a wave by DPP steps.
#pragma once

#include "common.h"

namespace moe {

// v of the lane that DPP control CTRL names (0 past the wave's ends: not reached here).
template <int CTRL, class T>
__device__ __forceinline__ T dpp(T v) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// After these four, a row of 16 lanes holds the same (op commutative, each lane's
// partner from the other half): quad_perm 1,0,3,2 and 2,3,0,1, row_half_mirror, row_mirror.
template <class T, class Op>
__device__ __forceinline__ T row_reduce(T v, const Op& op) {
  v = op(v, dpp<0xB1>(v));
  v = op(v, dpp<0x4E>(v));
  v = op(v, dpp<0x141>(v));
  return op(v, dpp<0x140>(v));
}
template <class T>
__device__ __forceinline__ T lane_of(T v, int lane) {
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, const Op& op) {
  v = row_reduce(v, op);
  return op(op(lane_of(v, 0), lane_of(v, 16)), op(lane_of(v, 32), lane_of(v, 48)));
}
}  // namespace moe
