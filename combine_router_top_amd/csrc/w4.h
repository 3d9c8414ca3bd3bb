// What the kernels of the 4-bit products share: their arguments, the rows of a
// segment, the masked or that makes bf16 numbers of packed values.  See expert_4bit.hip
// for the mathematics and the layout.
#pragma once

#include "common.h"
#include "kernels.h"
#include "seg_tile.h"

namespace moe {

constexpr int W4_KB = 128;   // K of a packed block

// Segments: rows [offsets[e], offsets[e+1]) of expert e, or, without offsets, one
// segment of rows [0, M).
struct W4Args {
  const bf16_t* a;         // [*][K]
  const char* b1;          // packed weights [n][ntiles][kb] blocks
  const char* b3;          // second matrix of a gated product
  const bf16_t* s1;        // [n][groups][N]
  const bf16_t* s3;
  const uint8_t* z1;       // [n][groups][N] or NULL
  const uint8_t* z3;
  void* c;                 // [*][N]
  const int32_t* offsets;
  int n, M;
  int K, N, kb, ntiles, groups;
  const int32_t* kr;       // tiles: exponents of the rows and of the columns [n][N]
  const int32_t* k1;
  const int32_t* k3;
  int parts, per;          // tiles: parts of K, and blocks of 128 K of each (the last may have fewer)
  int64_t part;            // bytes between the parts' products
};

__device__ __forceinline__ int w4_rows(const W4Args& p, int e, int& o) {
  int cnt = p.M;
  o = 0;
  if (p.offsets) {
    o = p.offsets[e];
    cnt = p.offsets[e + 1] - o;
  }
  o = __builtin_amdgcn_readfirstlane(o);
  cnt = __builtin_amdgcn_readfirstlane(cnt);
  return cnt;
}

// The eight numbers (16 + q) / 4096 of a packed word.  mask and bits are w4_mask() and w4_bits():
// as constants that the compiler knows they would be literals, of which a masked or
// takes none (then it is two instructions); it takes one scalar register.
__device__ __forceinline__ u32x4 w4_unpack(uint32_t w, uint32_t mask, uint32_t bits) {
  u32x4 o;
#pragma unroll
  for (int p = 0; p < 4; ++p) o[p] = ((p ? __builtin_amdgcn_alignbit(w, w, 4 * p) : w) & mask) | bits;
  return o;
}
__device__ __forceinline__ uint32_t w4_mask() {
  uint32_t v;
  asm("v_mov_b32 %0, 0x780078" : "=v"(v));
  return v;
}
__device__ __forceinline__ uint32_t w4_bits() {
  uint32_t v;
  asm("s_mov_b32 %0, 0x3B803B80" : "=s"(v));
  return v;
}

// expert_4bit_up.hip, expert_4bit_down.hip: the products on tiles, blocks of bm rows (64, 128
// or 192).  a: fp16 rows.
hipError_t launch_4bit_tiles_up(const W4Args& p, int group, int bm, int64_t rows_max, hipStream_t st);
hipError_t launch_4bit_tiles_down(const W4Args& p, int group, int bm, int64_t rows_max, bool f32out, hipStream_t st);

}  // namespace moe
