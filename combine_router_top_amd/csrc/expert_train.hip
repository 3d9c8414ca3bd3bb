// Training forward of the SwiGLU experts: the products of expert_gemm.hip, with
// the unactivated ones kept for the backward pass.
//
//   g = rnd(x W1), u = rnd(x W3), h = rnd(SiLU(x W1) (x W3)), y = rnd(h W2)
//
// bf16: two launches over the tiles of seg_tile.h; W1 and W3 products of an h
// column meet in one lane, so g, u and h leave from registers.  The launch pair
// of expert_gemm.hip streams a set of weight columns past at most 160 rows and would
// be faster where every segment is short (32 experts of 7168 x 2048, about 80 rows
// each: 485 against 545 us); where any segment is longer it reads those weights once
// more and in a second round of workgroups (about 128 rows each: 719 against 568 us;
// 16 .. 96 rows each, skewed: 735 against 570 .. 660 us).  Training batches are of
// that kind, and a host that knows the expected length alone cannot tell them apart, so
// the tiles take every size.
#include <stdint.h>

#include "common.h"
#include "f32_tile.h"
#include "kernels.h"
#include "seg_tile.h"

namespace moe {

int device_cus() {
  static const int n = [] {
    int dev = 0, c = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || c <= 0)
      c = 256;   // no device here: the part this is written for
    return c;
  }();
  return n;
}

template <int MT>
using UpCfg = StCfg<MT, ST_ROWS, ST_PANEL, f32x4, 1, true, 6 * MT, false, 256>;
template <int MT>
using DownCfg = StCfg<MT, ST_ROWS, ST_PANEL, f32x4, 1, false, 4 * MT, false, 256>;

// Both products of 128 h columns in one tile; W1 and W3 products of a column
// meet in a lane.  32 experts of about 128 rows, 7168 x 2048: 390 us, 5.0 TB/s; 2000
// rows of a dense block, 4104 x 1416: 69 us, the copy rate of 192 busy compute units.
template <int MT>
__global__ __launch_bounds__(ST_NT, 1) void keep_up_bf16(const bf16_t* __restrict__ x,
                                                         const int32_t* __restrict__ offsets, int n,
                                                         const bf16_t* __restrict__ w1,
                                                         const bf16_t* __restrict__ w3, bf16_t* __restrict__ g,
                                                         bf16_t* __restrict__ u, bf16_t* __restrict__ h, int d, int f,
                                                         int ntn) {
  using Cfg = UpCfg<MT>;
  __shared__ __attribute__((aligned(16))) char ring[Cfg::LDS];
  const int total = st_row_blocks(offsets, n, Cfg::BM) * ntn;
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  st_run<Cfg>(
      total, ring,
      [&](int L, StCtx<Cfg>& c) {
        const StTile t = st_tile_at(L, offsets, n, ntn, Cfg::BM);
        const int64_t eo = (int64_t)t.e * d * f;
        st_rows(c.a[0], x + (int64_t)t.r0 * d, (uint32_t)d * 2, t.R, (uint32_t)d * 2);
        st_panel(c.b[0], w1 + eo, (uint32_t)f * 2, d, 128 * t.nt, f, w3 + eo);
        c.nst = c.nst1 = (d + 63) / 64;
        return t;
      },
      [&](const StTile& t, typename Cfg::Acc& acc) {
        const int64_t first = (int64_t)t.r0 * f, ld = (int64_t)f * 2;
        const StOut og = st_out(g + first, ld, t.R), ou = st_out(u + first, ld, t.R), oh = st_out(h + first, ld, t.R);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int row = 16 * MT * (wave & 3) + 16 * mt + i;
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const int col = 128 * t.nt + 64 * (wave >> 2) + 16 * k + 8 * q;
            float x0[4], x1[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              x0[r] = silu_mul(acc[mt][k][r], acc[mt][k + 4][r]);
              x1[r] = silu_mul(acc[mt][k + 1][r], acc[mt][k + 5][r]);
            }
            st_put(og, row, 2u * (uint32_t)col, col < f, st_pack8(acc[mt][k], acc[mt][k + 1]));
            st_put(ou, row, 2u * (uint32_t)col, col < f, st_pack8(acc[mt][k + 4], acc[mt][k + 5]));
            st_put(oh, row, 2u * (uint32_t)col, col < f, st_pack8(x0, x1));
          }
        }
      });
}

template <int MT>
__global__ __launch_bounds__(ST_NT, 1) void keep_down_bf16(const bf16_t* __restrict__ h,
                                                           const int32_t* __restrict__ offsets, int n,
                                                           const bf16_t* __restrict__ w2, bf16_t* __restrict__ y,
                                                           int d, int f, int ntn) {
  using Cfg = DownCfg<MT>;
  __shared__ __attribute__((aligned(16))) char ring[Cfg::LDS];
  const int total = st_row_blocks(offsets, n, Cfg::BM) * ntn;
  st_run<Cfg>(
      total, ring,
      [&](int L, StCtx<Cfg>& c) {
        const StTile t = st_tile_at(L, offsets, n, ntn, Cfg::BM);
        st_rows(c.a[0], h + (int64_t)t.r0 * f, (uint32_t)f * 2, t.R, (uint32_t)f * 2);
        st_panel(c.b[0], w2 + (int64_t)t.e * f * d, (uint32_t)d * 2, f, 256 * t.nt, d);
        c.nst = c.nst1 = (f + 63) / 64;
        return t;
      },
      [&](const StTile& t, typename Cfg::Acc& acc) {
        const StOut o = st_out(y + (int64_t)t.r0 * d, (int64_t)d * 2, t.R);
        st_store_tile(o, acc, 256 * t.nt, d);
      });
}

__global__ __launch_bounds__(64 * F_NW) void keep_up_f32(const float* __restrict__ x, const int32_t* __restrict__ offsets,
                                                         int n, const float* __restrict__ w1,
                                                         const float* __restrict__ w3, float* __restrict__ g,
                                                         float* __restrict__ u, float* __restrict__ h, int d, int f) {
  __shared__ __attribute__((aligned(16))) F32Lds s;
  StTile t;
  if (!f32_row_block(offsets, n, blockIdx.x, t)) return;
  const int c0 = blockIdx.y * F_T;
  const float* a = x + (int64_t)t.r0 * d;
  const int64_t bo = (int64_t)t.e * d * f + c0;
  auto rows = [&](int k, int j) { return j < t.R ? a[(int64_t)j * d + k] : 0.f; };
  float acc[4][4] = {};
  f32_tile(rows, true, [&](int k, int j) { return c0 + j < f ? w1[bo + (int64_t)k * f + j] : 0.f; }, false, d, s, acc);
  const f32x2 gate = f32_join(s, acc);
  __syncthreads();   // the joined sums are read before the next slices arrive
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[p][r] = 0.f;
  f32_tile(rows, true, [&](int k, int j) { return c0 + j < f ? w3[bo + (int64_t)k * f + j] : 0.f; }, false, d, s, acc);
  const f32x2 up = f32_join(s, acc);
  const int row = f32_row(), col = c0 + f32_col();
  if (row >= t.R || col >= f) return;
  const int64_t at = (int64_t)(t.r0 + row) * f + col;
  f32x2 act;
#pragma unroll
  for (int r = 0; r < 2; ++r) act[r] = gate[r] / (1.0f + expf(-gate[r])) * up[r];
  *reinterpret_cast<f32x2*>(g + at) = gate;
  *reinterpret_cast<f32x2*>(u + at) = up;
  *reinterpret_cast<f32x2*>(h + at) = act;
}

__global__ __launch_bounds__(64 * F_NW) void keep_down_f32(const float* __restrict__ h, const int32_t* __restrict__ offsets,
                                                           int n, const float* __restrict__ w2, float* __restrict__ y,
                                                           int d, int f) {
  __shared__ __attribute__((aligned(16))) F32Lds s;
  StTile t;
  if (!f32_row_block(offsets, n, blockIdx.x, t)) return;
  const int c0 = blockIdx.y * F_T;
  const float* a = h + (int64_t)t.r0 * f;
  const float* b = w2 + (int64_t)t.e * f * d + c0;
  float acc[4][4] = {};
  f32_tile([&](int k, int j) { return j < t.R ? a[(int64_t)j * f + k] : 0.f; }, true,
           [&](int k, int j) { return c0 + j < d ? b[(int64_t)k * d + j] : 0.f; }, false, f, s, acc);
  const f32x2 v = f32_join(s, acc);
  const int row = f32_row(), col = c0 + f32_col();
  if (row < t.R && col < d) *reinterpret_cast<f32x2*>(y + (int64_t)(t.r0 + row) * d + col) = v;
}

hipError_t launch_expert_gemm_train(const Prob& p, const void* x_packed, const int32_t* offsets,
                                    const void* w1, const void* w3, const void* w2, void* g, void* u,
                                    void* h, void* y_packed, hipStream_t st) {
  if (p.dtype != 1) {
    const unsigned rb = f32_row_blocks(p);
    hipLaunchKernelGGL(keep_up_f32, dim3(rb, (p.f + F_T - 1) / F_T), dim3(64 * F_NW), 0, st, (const float*)x_packed,
                       offsets, p.n, (const float*)w1, (const float*)w3, (float*)g, (float*)u, (float*)h, p.d, p.f);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(keep_down_f32, dim3(rb, (p.d + F_T - 1) / F_T), dim3(64 * F_NW), 0, st, (const float*)h, offsets,
                       p.n, (const float*)w2, (float*)y_packed, p.d, p.f);
    return hipGetLastError();
  }
  const int nup = (p.f + 127) / 128, ndown = (p.d + 255) / 256;
  const TrainPlan plan = train_plan(device_cus(), p.tk(), p.E, p.n, p.d, p.f);
  hipError_t e = st_with_height(plan.up, [&](auto m) {
    hipLaunchKernelGGL(keep_up_bf16<m()>, st_row_grid(p.rows_max, p.n, m(), nup), dim3(ST_NT), 0, st,
                       (const bf16_t*)x_packed, offsets, p.n, (const bf16_t*)w1, (const bf16_t*)w3, (bf16_t*)g,
                       (bf16_t*)u, (bf16_t*)h, p.d, p.f, nup);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  return st_with_height(plan.down, [&](auto m) {
    hipLaunchKernelGGL(keep_down_bf16<m()>, st_row_grid(p.rows_max, p.n, m(), ndown), dim3(ST_NT), 0, st,
                       (const bf16_t*)h, offsets, p.n, (const bf16_t*)w2, (bf16_t*)y_packed, p.d, p.f, ndown);
    return hipGetLastError();
  });
}

}  // namespace moe
