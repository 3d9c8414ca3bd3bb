// fp32 products of the training calls: 32 x 32 tiles of eight waves that split K.
// The fp32 problems of this library are small and have tens of tiles, so what
// counts is how many trips to memory follow one another: each wave takes every
// eighth 16-deep slice of K through its own LDS, the next slice's operands loaded
// while one is multiplied, and the eight sums meet at the end, in a fixed order,
// every wave finishing an eighth of the tile.
#pragma once

#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "seg_tile.h"

namespace moe {

constexpr int F_K = 16, F_T = 32, F_LD = F_T + 4;   // slice depth, tile side, LDS row (16-byte aligned)
constexpr int F_NW = 8;                             // waves

struct F32Lds {
  float w[F_NW][2 * F_K * F_LD];   // a wave's slices of both operands, then its sums
};
static_assert(2 * F_K * F_LD >= F_T * F_T, "a wave's sums take the place of its slices");

// The first of the two neighbouring columns of this lane, and their row.
__device__ __forceinline__ int f32_row() { return 4 * ((threadIdx.x & 63) >> 3) + (threadIdx.x >> 7); }
__device__ __forceinline__ int f32_col() { return 4 * (threadIdx.x & 7) + 2 * ((threadIdx.x >> 6) & 1); }

// acc[p][r] of this lane: rows 4 ty + p, columns 4 tx + r (ty, tx = lane / 8,
// lane % 8) of this wave's part of the sum over k < K of A(k, row) B(k, column).
// A and B give 0 outside their operand; *_kfast: k is their contiguous index.
// All waves call.
template <class FA, class FB>
__device__ __forceinline__ void f32_tile(const FA& A, bool a_kfast, const FB& B, bool b_kfast, int K, F32Lds& s,
                                         float (&acc)[4][4]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tx = lane & 7, ty = lane >> 3;
  float* sa = s.w[wave];
  float* sb = sa + F_K * F_LD;
  float ra[8], rb[8];
  // element v of a lane: (k, j), the operand's contiguous index fastest over lanes
  auto kk = [&](bool kfast, int v) { return kfast ? lane & 15 : (lane >> 5) + 2 * v; };
  auto jj = [&](bool kfast, int v) { return kfast ? (lane >> 4) + 4 * v : lane & 31; };
  auto load = [&](int k0) {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const int ka = k0 + kk(a_kfast, v), kb = k0 + kk(b_kfast, v);
      ra[v] = ka < K ? A(ka, jj(a_kfast, v)) : 0.f;
      rb[v] = kb < K ? B(kb, jj(b_kfast, v)) : 0.f;
    }
  };
  load(F_K * wave);
  for (int k0 = F_K * wave; k0 < K; k0 += F_NW * F_K) {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      sa[kk(a_kfast, v) * F_LD + jj(a_kfast, v)] = ra[v];
      sb[kk(b_kfast, v) * F_LD + jj(b_kfast, v)] = rb[v];
    }
    lds_wave_order();   // this wave alone writes and reads its part
    if (k0 + F_NW * F_K < K) load(k0 + F_NW * F_K);
#pragma unroll
    for (int k = 0; k < F_K; ++k) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(sa + k * F_LD + 4 * ty);
      const f32x4 b = *reinterpret_cast<const f32x4*>(sb + k * F_LD + 4 * tx);
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[p][r] = fmaf(a[p], b[r], acc[p][r]);
    }
    lds_wave_order();
  }
}

// The waves' sums added, in their order: this lane's two values, at f32_row() and
// f32_col().  All waves call; LDS may be written again after a barrier.
__device__ __forceinline__ f32x2 f32_join(F32Lds& s, const float (&acc)[4][4]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int r = 0; r < 4; ++r) s.w[wave][(4 * p + r) * 64 + lane] = acc[p][r];
  __syncthreads();
  f32x2 v = {0.f, 0.f};
#pragma unroll
  for (int w = 0; w < F_NW; ++w) {
    v[0] += s.w[w][2 * wave * 64 + lane];
    v[1] += s.w[w][(2 * wave + 1) * 64 + lane];
  }
  return v;
}

// Row block b of 32 rows, counted over all segments; false past the last.
__device__ __forceinline__ bool f32_row_block(const int32_t* offsets, int n, int b, StTile& t) {
  t = st_tile_at(b, offsets, n, 1, F_T);
  return t.R > 0;
}

// At most this many blocks of 32 rows, over all segments.
inline unsigned f32_row_blocks(const Prob& p) {
  return (unsigned)std::min<int64_t>((p.rows_max + F_T - 1) / F_T + p.n, p.rows_max);
}

}  // namespace moe
