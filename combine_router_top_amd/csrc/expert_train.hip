// Training forward of the SwiGLU experts: the products of expert_gemm.hip, with
// the unactivated ones kept for the backward pass.
//
//   g = rnd(x W1), u = rnd(x W3), h = rnd(SiLU(x W1) (x W3)), y = rnd(h W2)
//
// Three regimes.  Where the weights' stream bounds the pass (tens to a few
// hundred rows an expert, large weights) the streaming kernels of
// expert_gemm.hip run with an epilogue that also stores g and u: a workgroup
// there reads 512 weight columns for at most 160 rows.  Long segments (dense
// routing, a dense block) and small problems take the tiles of seg_tile.h: the
// former because the matrix cores bound them, the latter because those tiles
// come small enough to occupy the compute units.
#include <stdint.h>

#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "seg_tile.h"

namespace moe {

template <int MT>
using UpCfg = StCfg<MT, ST_ROWS, ST_PANEL, f32x4, 1, true, 6 * MT, false, 256>;
template <int MT>
using DownCfg = StCfg<MT, ST_ROWS, ST_PANEL, f32x4, 1, false, 4 * MT, false, 256>;

// Both products of 128 h columns in one tile; W1 and W3 products of a column
// meet in a lane.
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

hipError_t launch_expert_gemm_train(const Prob& p, const void* x_packed, const int32_t* offsets,
                                    const void* w1, const void* w3, const void* w2, void* g, void* u,
                                    void* h, void* y_packed, void* ws, hipStream_t st) {
  const int64_t mean = p.tk() / p.E;
  const int nup = (p.f + 127) / 128, ndown = (p.d + 255) / 256;
  const int64_t small = (int64_t)p.n * std::max<int64_t>(1, (mean + 63) / 64) * std::max(nup, ndown);
  const int cus = device_cus();
  const bool wide = p.d > (1 << 20) || p.f > (1 << 20);   // beyond seg_tile.h's 32-bit offsets
  if (p.dtype != 1 || wide || (mean < 320 && small > cus))
    return launch_expert_gemm_keep(p, x_packed, offsets, w1, w3, w2, g, u, h, y_packed, ws, st);
  const int64_t seg = std::max<int64_t>(1, mean);
  hipError_t e = st_with_height(
      st_height(p.n, seg, (p.d + 63) / 64, {0, nup, nup, nup, nup}, {0, 256, 256, 256, 256}), [&](auto m) {
        hipLaunchKernelGGL(keep_up_bf16<m()>, st_row_grid(p.rows_max, p.n, m(), nup), dim3(ST_NT), 0, st,
                           (const bf16_t*)x_packed, offsets, p.n, (const bf16_t*)w1, (const bf16_t*)w3, (bf16_t*)g,
                           (bf16_t*)u, (bf16_t*)h, p.d, p.f, nup);
        return hipGetLastError();
      });
  if (e != hipSuccess) return e;
  return st_with_height(st_height(p.n, seg, (int64_t)p.f * 2, p.d, 256), [&](auto m) {
    hipLaunchKernelGGL(keep_down_bf16<m()>, st_row_grid(p.rows_max, p.n, m(), ndown), dim3(ST_NT), 0, st,
                       (const bf16_t*)h, offsets, p.n, (const bf16_t*)w2, (bf16_t*)y_packed, p.d, p.f, ndown);
    return hipGetLastError();
  });
}

}  // namespace moe
