// Backward pass of the SwiGLU expert FFNs over expert-contiguous segments.  For
// the rows R of expert e, with g = x W1, u = x W3, h = SiLU(g) u as the forward
// pass kept them and s = 1 / (1 + exp(-g)):
//
//   dh    = dy W2^T                           (fp32, never stored)
//   dg    = rnd(dh u s (1 + g (1 - s)))       du = rnd(dh g s)
//   dx    = rnd(dg W1^T + du W3^T)            (one fp32 sum over both products)
//   dW1_e = rnd(x^T dg), dW3_e = rnd(x^T du), dW2_e = rnd(h^T dy)
//
// Two launches: the gate gradient (dh with its epilogue), then the input gradient
// and all weight gradients.  The one rounding inside is that of dg and du to
// the storage type, which the matrix cores need of their operands: in bf16 it costs
// up to 2^-8 relative once per value, as the rounding of h does in the forward pass;
// in fp32 there is none.  Every other sum stays in fp32.
//
// bf16: tiles of seg_tile.h.  The first two products contract over a dimension
// that both operands hold contiguously (dy and rows of W2; dg and rows of W1),
// the weight gradients over a segment's rows, which neither does: there both
// operands are read as panels and transposed by the LDS read.  No operand is
// ever transposed in memory.
#include <stdint.h>

#include <algorithm>

#include "common.h"
#include "f32_tile.h"
#include "kernels.h"
#include "seg_tile.h"

namespace moe {

// d/dg and d/du of SiLU(g) u, times dh.  The hardware exponential and
// reciprocal as in silu_mul; both limits of g are exact (s = 0 or 1).
__device__ __forceinline__ void swiglu_grad(float dh, float g, float u, float& dg, float& du) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
  dg = dh * u * (s * fmaf(g, 1.0f - s, 1.0f));
  du = dh * (g * s);
}

template <int MT>
using GateCfg = StCfg<MT, ST_ROWS, ST_ROWS, f32x4, 1, false, (MT == 1 ? 4 : 8) * MT>;
template <int MT>
using InputCfg = StCfg<MT, ST_ROWS, ST_ROWS, f32x4, 2, false, (MT == 1 ? 2 : 4) * MT, false, MT == 1 ? 128 : 256, MT != 4>;
template <int MODE>
using WeightCfg = StCfg<4, ST_PANEL, ST_PANEL, f32x4, 1, false, MODE == WG_SPLIT ? 32 : 16, MODE == WG_SHORT>;

// dh tiles: rows of dy against rows of W2 (its f rows are the output columns).
// 32 experts of about 128 rows, 7168 x 2048: 206 us, 4.6 TB/s of weights, read in
// pieces of 128 bytes a row; 8 dense experts 4096 x 14336, 32768 rows: 3.45 ms, 1.12
// PFLOP/s.
template <int MT>
__global__ __launch_bounds__(ST_NT, 1) void gate_grad_bf16(const bf16_t* __restrict__ dy,
                                                           const int32_t* __restrict__ offsets, int n,
                                                           const bf16_t* __restrict__ w2,
                                                           const bf16_t* __restrict__ g,
                                                           const bf16_t* __restrict__ u,
                                                           bf16_t* __restrict__ dg, bf16_t* __restrict__ du,
                                                           int d, int f, int ntn) {
  using Cfg = GateCfg<MT>;
  __shared__ __attribute__((aligned(16))) char ring[Cfg::LDS];
  const int total = st_row_blocks(offsets, n, Cfg::BM) * ntn;
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 3, wn = wave >> 2;
  st_run<Cfg>(
      total, ring,
      [&](int L, StCtx<Cfg>& c) {
        const StTile t = st_tile_at(L, offsets, n, ntn, Cfg::BM);
        const uint32_t ld = (uint32_t)d * 2;
        st_rows(c.a[0], dy + (int64_t)t.r0 * d, ld, t.R, ld);
        st_rows(c.b[0], w2 + ((int64_t)t.e * f + Cfg::BN * t.nt) * d, ld, min(Cfg::BN, f - Cfg::BN * t.nt), ld);
        c.nst = c.nst1 = (d + 63) / 64;
        return t;
      },
      [&](const StTile& t, typename Cfg::Acc& acc) {
        const int64_t first = (int64_t)t.r0 * f;
        const int64_t ld = (int64_t)f * 2;
        const StOut og = st_out(dg + first, ld, t.R), ou = st_out(du + first, ld, t.R);
        const __amdgpu_buffer_rsrc_t rg = gc_rsrc(g + first, (uint32_t)t.R * (uint32_t)ld);
        const __amdgpu_buffer_rsrc_t ru = gc_rsrc(u + first, (uint32_t)t.R * (uint32_t)ld);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int row = 16 * MT * wm + 16 * mt + i;
          u32x4 gv[Cfg::NT / 2], uv[Cfg::NT / 2];
#pragma unroll
          for (int k = 0; k < Cfg::NT / 2; ++k) {
            const int col = Cfg::BN * t.nt + Cfg::WN * wn + 32 * k + 8 * q;
            const uint32_t at = col < f ? (uint32_t)row * (uint32_t)ld + 2u * (uint32_t)col : 0xFFFFFFF0u;
            gv[k] = __builtin_amdgcn_raw_buffer_load_b128(rg, at, 0, 0);
            uv[k] = __builtin_amdgcn_raw_buffer_load_b128(ru, at, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < Cfg::NT / 2; ++k) {
            const int col = Cfg::BN * t.nt + Cfg::WN * wn + 32 * k + 8 * q;
            float x[4], y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              x[r] = acc[mt][2 * k][r];
              y[r] = acc[mt][2 * k + 1][r];
              st_swap_pair(x[r], y[r]);   // x: columns 8 q + r, y: 8 q + 4 + r
            }
            u32x4 vg, vu;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const float* dh = h < 2 ? x + 2 * h : y + 2 * (h - 2);
              float a0, a1, b0, b1;
              swiglu_grad(dh[0], bf16_lo(gv[k][h]), bf16_lo(uv[k][h]), a0, b0);
              swiglu_grad(dh[1], bf16_hi(gv[k][h]), bf16_hi(uv[k][h]), a1, b1);
              vg[h] = cvt_bf16x2(a0, a1);
              vu[h] = cvt_bf16x2(b0, b1);
            }
            st_put(og, row, 2u * (uint32_t)col, col < f, vg);
            st_put(ou, row, 2u * (uint32_t)col, col < f, vu);
          }
        }
      });
}

// A finished tile through a 4 KB staging area of each wave: a store then writes four
// rows of 256 bytes instead of sixteen pieces of 64, which cost the address
// unit about 100 cycles an instruction and bounded tiles that mostly store.
// Staged rows keep their 32-byte chunk c at c ^ (row & 7), rows 8 .. 15 with its
// halves exchanged, so that 32 lanes' writes meet 64 distinct banks (sparse
// weight gradients 825 -> 789 us).  The stores pass L2 by, except for narrow rows
// that do not start on cache lines, whose pieces L2 merges (30 experts of 64 rows,
// rows of 784 bytes: 378 -> 313 us; of 768: 237 past L2, 269 through it; four
// column blocks of 2000 bytes: 142 and 171).  Where exactly wider rows change sides is
// not known: with M = 7168 and 30 experts of 64 rows, going through L2 was faster up to
// the widest tried (rows of 976 bytes 412 past, 354 through; 1040: 487, 450; 1424:
// 613, 521; 2000: 778, 682; 2448: 997, 892).
__device__ __forceinline__ void store_tile_rows(const StOut& o, const f32x4 (&acc)[4][8], int col0, int N, char* stage) {
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char* stg = stage + 4096 * wave;
  const bool merge = N <= 512 && (N & 63) != 0;
  const int p = lane & 15, col = col0 + 128 * (wave >> 2) + 8 * p;
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const f32x4 v = acc[mt][t];
      *reinterpret_cast<u32x2*>(stg + i * 256 + 32 * (t ^ (i & 7)) + 8 * (q ^ (2 * (i >> 3)))) =
          u32x2{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
    }
    lds_wave_order();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 4 * k + q;
      const u32x4 v = *reinterpret_cast<const u32x4*>(stg + row * 256 + 32 * ((p >> 1) ^ (row & 7)) + 16 * ((p & 1) ^ (row >> 3)));
      if (merge) st_put(o, 64 * (wave & 3) + 16 * mt + row, 2u * (uint32_t)col, col < N, v);
      else st_put<true>(o, 64 * (wave & 3) + 16 * mt + row, 2u * (uint32_t)col, col < N, v);
    }
    lds_wave_order();
  }
}

// The input gradient (8 dense experts: 6.2 ms, 1.24 PFLOP/s): [dg | du] against rows of W1, then of W3, in one accumulator.
struct InputGrad {
  const bf16_t* dg;
  const bf16_t* du;
  const bf16_t* w1;
  const bf16_t* w3;
  bf16_t* dx;   // NULL: not wanted
  int d, f, ntn;
};

// Its tiles; returns their number.
template <int MT>
__device__ __forceinline__ int input_tiles(const InputGrad& p, const int32_t* __restrict__ offsets, int n, char* ring) {
  using Cfg = InputCfg<MT>;
  if (!p.dx) return 0;
  const bf16_t* __restrict__ dg = p.dg;
  const bf16_t* __restrict__ du = p.du;
  const bf16_t* __restrict__ w1 = p.w1;
  const bf16_t* __restrict__ w3 = p.w3;
  bf16_t* __restrict__ dx = p.dx;
  const int d = p.d, f = p.f, ntn = p.ntn;
  const int total = st_row_blocks(offsets, n, Cfg::BM) * ntn;
  st_run<Cfg>(
      total, ring,
      [&](int L, StCtx<Cfg>& c) {
        const StTile t = st_tile_at(L, offsets, n, ntn, Cfg::BM);
        const uint32_t ld = (uint32_t)f * 2;
        const int64_t arow = (int64_t)t.r0 * f, brow = ((int64_t)t.e * d + Cfg::BN * t.nt) * f;
        const int cols = min(Cfg::BN, d - Cfg::BN * t.nt);
        st_rows(c.a[0], dg + arow, ld, t.R, ld);
        st_rows(c.a[1], du + arow, ld, t.R, ld);
        st_rows(c.b[0], w1 + brow, ld, cols, ld);
        st_rows(c.b[1], w3 + brow, ld, cols, ld);
        c.nst1 = (f + 63) / 64;
        c.nst = 2 * c.nst1;
        // Rows a multiple of 4 KB apart: all rows' pieces of one stage lie in a few
        // memory channels, and workgroups that run in step all read the same
        // stage.  Each starts at another one (32 experts of 128 rows, 4 KB rows:
        // 470 -> 428 us; with rows of other lengths it only costs L2 hits, as it
        // does where long segments share weight columns).
        c.rot = Cfg::ROT && (ld & 4095) == 0 ? (int)(blockIdx.x >> 3) % c.nst : 0;
        return t;
      },
      [&](const StTile& t, typename Cfg::Acc& acc) {
        st_store_tile(st_out(dx + (int64_t)t.r0 * d, (int64_t)d * 2, t.R), acc, Cfg::BN * t.nt, d);
      });
  return total;
}

// One weight gradient C_e [M][N] = P^T Q over the segment's rows, P [rows][M],
// Q [rows][N].
struct WeightGrad {
  const bf16_t* P;
  const bf16_t* Q;
  bf16_t* C;
  int M, N;
};
struct WeightGrads {
  WeightGrad m[3];
};

// All tiles of all wanted weight gradients, expert by expert (8 dense experts: 9.1
// ms, 1.27 PFLOP/s); a segment without rows gives zeros.  WG_SHORT: units of at most `div` row blocks.  WG_SPLIT: each
// tile's rows go to `div` workgroups, whose fp32 sums m[].C holds as [div][n][M][N].
// first: this workgroup's first tile (unit).
template <int MODE>
__device__ __forceinline__ void weight_tiles(const WeightGrads& w, int nm, int div, const int32_t* __restrict__ offsets,
                                             int n, char* ring, int start) {
  using Cfg = WeightCfg<MODE>;
  constexpr bool SHORT = MODE == WG_SHORT;
  // the table as values: a choice between its addresses would put it in scratch,
  // and what is read from there into vector registers
  auto held = [&](WeightGrad m) {
    asm volatile("" : "+s"(m.P), "+s"(m.Q), "+s"(m.C), "+s"(m.M), "+s"(m.N));
    return m;
  };
  const WeightGrad m0 = held(w.m[0]), m1 = held(w.m[1]), m2 = held(w.m[2]);
  // column blocks, runs of row blocks and their length, and the tiles (SHORT:
  // units) of each matrix
  auto runs_of = [&](int M) { return max(1, SHORT ? st_div((M + 255) / 256 + div - 1, div) : (M + 255) / 256); };
  auto len_of = [&](int M, int runs) { return st_div((M + 255) / 256 + runs - 1, runs); };
  const int r0 = runs_of(m0.M), r1 = runs_of(m1.M), r2 = runs_of(m2.M);
  const int l0 = len_of(m0.M, r0), l1 = len_of(m1.M, r1), l2 = len_of(m2.M, r2);
  const int n0 = (m0.N + 255) / 256, n1 = (m1.N + 255) / 256, n2 = (m2.N + 255) / 256;
  const int c0 = n0 * r0, c1 = nm > 1 ? n1 * r1 : 0, c2 = nm > 2 ? n2 * r2 : 0;
  const int all = c0 + c1 + c2, per = MODE == WG_SPLIT ? div * all : all;
  struct Unit {
    WeightGrad m;
    int e, tm, tn, tiles;   // row blocks tm .. tm + tiles - 1
    int o, cnt, nst, part;   // part (WG_SPLIT): which share of the rows
  };
  auto unit = [&](int L) __attribute__((always_inline)) {
    Unit r;
    r.e = st_div(L, per);
    int at = L - r.e * per;
    r.part = MODE == WG_SPLIT ? st_div(at, all) : 0;
    at -= r.part * all;
    const bool b1 = at >= c0, b2 = at >= c0 + c1;
    auto pick = [&](auto v0, auto v1, auto v2) { return b2 ? v2 : b1 ? v1 : v0; };
    at -= pick(0, c0, c0 + c1);
    r.m.P = pick(m0.P, m1.P, m2.P);
    r.m.Q = pick(m0.Q, m1.Q, m2.Q);
    r.m.C = pick(m0.C, m1.C, m2.C);
    r.m.M = pick(m0.M, m1.M, m2.M);
    r.m.N = pick(m0.N, m1.N, m2.N);
    const int nnt = pick(n0, n1, n2);
    if (SHORT) {
      // the column blocks of the same rows run together, so that whole rows of
      // the gradient are written at a time
      const int q = st_div(at, nnt), ln = pick(l0, l1, l2);
      r.tn = at - q * nnt;
      r.tm = q * ln;
      r.tiles = min(ln, (r.m.M + 255) / 256 - r.tm);
    } else {
      // groups of 8 row blocks run through the columns together
      const int mg = st_div(at, ST_GM * nnt), rem = at - mg * ST_GM * nnt;
      const int gsz = min(ST_GM, (r.m.M + 255) / 256 - mg * ST_GM);
      r.tn = st_div(rem, gsz);
      r.tm = mg * ST_GM + (rem - r.tn * gsz);
      r.tiles = 1;
    }
    r.o = __builtin_amdgcn_readfirstlane(offsets[r.e]);
    r.cnt = __builtin_amdgcn_readfirstlane(offsets[r.e + 1]) - r.o;
    r.nst = (r.cnt + 63) / 64;
    if (SHORT && r.nst == 1) r.nst = 2;
    if (MODE == WG_SPLIT) {   // an equal share of the stages; the last ones may be empty
      const int share = st_div(r.nst + div - 1, div), first = 64 * share * r.part;
      r.o += first;
      r.cnt = max(0, min(r.cnt - first, 64 * share));
      r.nst = (r.cnt + 63) / 64;
    }
    return r;
  };
  auto cols = [&](const Unit& r, StCtx<Cfg>& c) __attribute__((always_inline)) {
    st_panel(c.b[0], r.m.Q + (int64_t)r.o * r.m.N, (uint32_t)r.m.N * 2, r.cnt, 256 * r.tn, r.m.N);
    c.nst = c.nst1 = r.nst;
  };
  auto rows = [&](const Unit& r, int j, StCtx<Cfg>& c) __attribute__((always_inline)) {
    st_panel(c.a[0], r.m.P + (int64_t)r.o * r.m.M, (uint32_t)r.m.M * 2, r.cnt, 256 * (r.tm + j), r.m.M);
  };
  auto out = [&](const Unit& r, int j) {
    const int row = 256 * (r.tm + j);
    return st_out(r.m.C + ((int64_t)r.e * r.m.M + row) * r.m.N, (int64_t)r.m.N * 2, min(256, r.m.M - row));
  };
  if constexpr (SHORT) {
    st_run_short<Cfg>(n * per, ring, unit, cols, rows, [&](const Unit& r, int j, f32x4 (&acc)[4][8]) {
      store_tile_rows(out(r, j), acc, 256 * r.tn, r.m.N, ring + Cfg::LDS);
    }, start);
  } else {
    st_run<Cfg>(
        n * per, ring,
        [&](int L, StCtx<Cfg>& c) {
          const Unit r = unit(L);
          cols(r, c);
          rows(r, 0, c);
          return r;
        },
        [&](const Unit& r, f32x4 (&acc)[4][8]) {
          if constexpr (MODE == WG_SPLIT) {
            const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const int row0 = 256 * r.tm;
            float* C = reinterpret_cast<float*>(r.m.C) + (((int64_t)r.part * n + r.e) * r.m.M + row0) * r.m.N;
            const StOut o = st_out(C, (int64_t)r.m.N * 4, min(256, r.m.M - row0));
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
              for (int t = 0; t < 8; ++t) {
                const int col = 256 * r.tn + 128 * (wave >> 2) + 16 * t + 4 * (lane >> 4);
                st_put(o, 64 * (wave & 3) + 16 * mt + (lane & 15), 4u * (uint32_t)col, col < r.m.N,
                       __builtin_bit_cast(u32x4, acc[mt][t]));
              }
          } else {
            st_store_tile(out(r, 0), acc, 256 * r.tn, r.m.N);
          }
        },
        start);
  }
}

// Both in one launch: neither needs the other, and in small problems neither has a
// tile for every compute unit (backward pass of 64 tokens, 4 experts of 512 x 512
// 28.5 -> 20.8 us, one token and 8 experts of 2048 x 1024 59 -> 50, 32 x 128 rows
// 1445 -> 1430).
template <int MT, int MODE>
__global__ __launch_bounds__(ST_NT, 1) void input_weight_grad_bf16(InputGrad in, WeightGrads w, int nm, int div,
                                                                   const int32_t* __restrict__ offsets, int n) {
  constexpr int LI = InputCfg<MT>::LDS, LW = WeightCfg<MODE>::LDS + (MODE == WG_SHORT ? 8 * 4096 : 0);
  __shared__ __attribute__((aligned(16))) char ring[LI > LW ? LI : LW];
  const int before = input_tiles<MT>(in, offsets, n, ring);
  if (nm) weight_tiles<MODE>(w, nm, div, offsets, n, ring, st_second_tile(before));
}

// C = rnd(sum of the `div` parts), in their order; blockIdx.y is the matrix.
struct WeightSums {
  const float* part[3];
  bf16_t* C[3];
};
__global__ __launch_bounds__(256) void weight_grad_sum(WeightSums w, int div, int64_t count) {
  const float* p = w.part[blockIdx.y];
  const int64_t n8 = count / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    f32x4 a = reinterpret_cast<const f32x4*>(p)[2 * i], b = reinterpret_cast<const f32x4*>(p)[2 * i + 1];
    for (int s = 1; s < div; ++s) {
      const f32x4* q = reinterpret_cast<const f32x4*>(p + s * count) + 2 * i;
      a += q[0];
      b += q[1];
    }
    reinterpret_cast<u32x4*>(w.C[blockIdx.y])[i] =
        u32x4{cvt_bf16x2(a[0], a[1]), cvt_bf16x2(a[2], a[3]), cvt_bf16x2(b[0], b[1]), cvt_bf16x2(b[2], b[3])};
  }
}

// fp32: f32_tile.h
__global__ __launch_bounds__(64 * F_NW) void gate_grad_f32(const float* __restrict__ dy, const int32_t* __restrict__ offsets,
                                                     int n, const float* __restrict__ w2, const float* __restrict__ g,
                                                     const float* __restrict__ u, float* __restrict__ dg,
                                                     float* __restrict__ du, int d, int f) {
  __shared__ __attribute__((aligned(16))) F32Lds s;
  StTile t;
  if (!f32_row_block(offsets, n, blockIdx.x, t)) return;
  const int c0 = blockIdx.y * F_T;
  const float* a = dy + (int64_t)t.r0 * d;
  const float* b = w2 + ((int64_t)t.e * f + c0) * d;
  // g and u of this lane's values, on their way while the product runs
  const int row = f32_row(), col = c0 + f32_col();
  const bool live = row < t.R && col < f;
  const int64_t at = (int64_t)(t.r0 + row) * f + col;
  f32x2 gv = {0.f, 0.f}, uv = {0.f, 0.f};
  if (live) {
    gv = *reinterpret_cast<const f32x2*>(g + at);
    uv = *reinterpret_cast<const f32x2*>(u + at);
  }
  float acc[4][4] = {};
  f32_tile([&](int k, int j) { return j < t.R ? a[(int64_t)j * d + k] : 0.f; }, true,
           [&](int k, int j) { return c0 + j < f ? b[(int64_t)j * d + k] : 0.f; }, true, d, s, acc);
  const f32x2 dh = f32_join(s, acc);
  if (!live) return;
  f32x2 vg, vu;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float sg = 1.0f / (1.0f + expf(-gv[r]));
    vg[r] = dh[r] * uv[r] * (sg * (1.0f + gv[r] * (1.0f - sg)));
    vu[r] = dh[r] * (gv[r] * sg);
  }
  *reinterpret_cast<f32x2*>(dg + at) = vg;
  *reinterpret_cast<f32x2*>(du + at) = vu;
}

// The input and weight gradients that are wanted: C_e [M][N] = P^T Q over the
// segment's rows for up to three matrices, and dx; a 32 x 32 tile for each workgroup,
// in one launch (64 tokens, 8 experts of 128 x 256: whole pass 33.7 -> 17.5 us with
// the shared join and the gate's early loads).
struct GradsF32 {
  const float* dg;
  const float* du;
  const float* w1;
  const float* w3;
  float* dx;
  int d, f;
  int64_t in_tiles;   // row blocks * ceil(d / 32), or 0
  int row_blocks;
  struct {
    const float* P;
    const float* Q;
    float* C;
    int M, N;
  } m[3];
  int nm;
  int64_t tiles;      // in_tiles + n * nm * ceil(d / 32) * ceil(f / 32)
};

__device__ __forceinline__ void input_tile_f32(const GradsF32& p, int64_t tile, const int32_t* __restrict__ offsets,
                                               int n, F32Lds& s) {
  const int d = p.d, f = p.f;
  StTile t;
  const int c = (int)(tile / p.row_blocks);
  if (!f32_row_block(offsets, n, (int)(tile - (int64_t)c * p.row_blocks), t)) return;
  const int c0 = c * F_T;
  const int64_t ar = (int64_t)t.r0 * f, br = ((int64_t)t.e * d + c0) * f;
  float acc[4][4] = {};
  // both products as one sum over 2 f
  f32_tile([&](int k, int j) { return j < t.R ? (k < f ? p.dg + ar : p.du + ar - f)[(int64_t)j * f + k] : 0.f; }, true,
           [&](int k, int j) { return c0 + j < d ? (k < f ? p.w1 + br : p.w3 + br - f)[(int64_t)j * f + k] : 0.f; }, true,
           2 * f, s, acc);
  const f32x2 v = f32_join(s, acc);
  const int row = f32_row(), col = c0 + f32_col();
  if (row < t.R && col < d) *reinterpret_cast<f32x2*>(p.dx + (int64_t)(t.r0 + row) * d + col) = v;
}

__device__ __forceinline__ void weight_tile_f32(const GradsF32& p, int64_t tile, const int32_t* __restrict__ offsets,
                                                F32Lds& s) {
  const int64_t each = (p.tiles - p.in_tiles) / p.nm;   // n * tiles of a matrix, alike for all of them
  const int k0 = (int)(tile / each);
  const auto m = k0 == 0 ? p.m[0] : k0 == 1 ? p.m[1] : p.m[2];
  tile -= k0 * each;
  const int nm = (m.M + F_T - 1) / F_T, nn = (m.N + F_T - 1) / F_T;
  const int e = (int)(tile / ((int64_t)nm * nn)), at = (int)(tile - (int64_t)e * nm * nn);
  const int m0 = at / nn * F_T, n0 = at % nn * F_T;
  const int o = offsets[e], cnt = offsets[e + 1] - o;
  const float* a = m.P + (int64_t)o * m.M + m0;
  const float* b = m.Q + (int64_t)o * m.N + n0;
  float acc[4][4] = {};
  f32_tile([&](int k, int j) { return m0 + j < m.M ? a[(int64_t)k * m.M + j] : 0.f; }, false,
           [&](int k, int j) { return n0 + j < m.N ? b[(int64_t)k * m.N + j] : 0.f; }, false, cnt, s, acc);
  const f32x2 v = f32_join(s, acc);
  const int row = m0 + f32_row(), col = n0 + f32_col();
  if (row < m.M && col < m.N) *reinterpret_cast<f32x2*>(m.C + ((int64_t)e * m.M + row) * m.N + col) = v;
}

__global__ __launch_bounds__(64 * F_NW) void input_weight_grad_f32(GradsF32 p, const int32_t* __restrict__ offsets, int n) {
  __shared__ __attribute__((aligned(16))) F32Lds s;
  const int64_t tile = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (tile < p.in_tiles) input_tile_f32(p, tile, offsets, n, s);
  else if (tile < p.tiles) weight_tile_f32(p, tile - p.in_tiles, offsets, s);
}

// Zeros (the weight gradients of an empty batch): a kernel, so that a captured
// call holds no memset node.
__global__ __launch_bounds__(256) void fill_zero(u32x4* __restrict__ p, int64_t n16) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += (int64_t)gridDim.x * 256)
    p[i] = u32x4{0u, 0u, 0u, 0u};
}

static size_t pad256(size_t v) { return (v + 255) / 256 * 256; }

size_t expert_backward_ws_bytes(const Prob& p) {
  // dg and du, [rows_max, f] each, and the parts of split weight gradients
  const int parts = p.dtype == 1 && p.T > 0 ? weight_parts(device_cus(), p.tk(), p.E, p.n, p.d, p.f) : 1;
  return 2 * pad256((size_t)p.rows_max * p.f * p.elem()) +
         (parts > 1 ? 3 * pad256((size_t)parts * p.n * p.d * p.f * 4) : 0);
}

hipError_t launch_expert_backward(const Prob& p, const void* x, const int32_t* offsets, const void* w1,
                                  const void* w3, const void* w2, const void* g, const void* u, const void* h,
                                  const void* dy, void* dx, void* dw1, void* dw3, void* dw2, void* ws,
                                  hipStream_t st) {
  hipError_t e;
  if (p.T == 0) {
    const int64_t n16 = (int64_t)p.n * p.d * p.f * p.elem() / 16;
    for (void* w : {dw1, dw3, dw2}) {
      if (!w) continue;
      hipLaunchKernelGGL(fill_zero, dim3((unsigned)std::min<int64_t>((n16 + 255) / 256, 2048)), dim3(256), 0, st,
                         (u32x4*)w, n16);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
  }
  char* dgp = (char*)ws;
  char* dup = dgp + pad256((size_t)p.rows_max * p.f * p.elem());
  const bool gate = dx || dw1 || dw3;
  if (p.dtype != 1) {
    const unsigned rb = f32_row_blocks(p);
    const unsigned cf = (unsigned)((p.f + F_T - 1) / F_T), cd = (unsigned)((p.d + F_T - 1) / F_T);
    if (gate) {
      hipLaunchKernelGGL(gate_grad_f32, dim3(rb, cf), dim3(64 * F_NW), 0, st, (const float*)dy, offsets, p.n,
                         (const float*)w2, (const float*)g, (const float*)u, (float*)dgp, (float*)dup, p.d, p.f);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    GradsF32 q{(const float*)dgp, (const float*)dup, (const float*)w1, (const float*)w3, (float*)dx, p.d, p.f};
    q.row_blocks = (int)rb;
    q.in_tiles = dx ? (int64_t)rb * cd : 0;
    q.tiles = q.in_tiles;
    auto want = [&](const void* P, const void* Q, void* C, int M, int N) {
      if (!C) return;
      auto& m = q.m[q.nm++];
      m.P = (const float*)P;
      m.Q = (const float*)Q;
      m.C = (float*)C;
      m.M = M;
      m.N = N;
      q.tiles += (int64_t)p.n * cd * cf;
    };
    want(x, dgp, dw1, p.d, p.f);
    want(x, dup, dw3, p.d, p.f);
    want(h, dy, dw2, p.f, p.d);
    if (q.tiles) {
      const int64_t gx = std::min<int64_t>(q.tiles, 1 << 16);
      hipLaunchKernelGGL(input_weight_grad_f32, dim3((unsigned)gx, (unsigned)((q.tiles + gx - 1) / gx)), dim3(64 * F_NW),
                         0, st, q, offsets, p.n);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const BackwardPlan plan =
      backward_plan(device_cus(), p.tk(), p.E, p.n, p.d, p.f, dx, (dw1 != nullptr) + (dw3 != nullptr) + (dw2 != nullptr));
  const bf16_t* DG = (const bf16_t*)dgp;
  const bf16_t* DU = (const bf16_t*)dup;
  if (gate) {
    e = st_with_height(plan.gate, [&](auto h) {
      constexpr int bn = GateCfg<h()>::BN;
      const int ntn = (p.f + bn - 1) / bn;
      hipLaunchKernelGGL(gate_grad_bf16<h()>, st_row_grid(p.rows_max, p.n, h(), ntn), dim3(ST_NT), 0, st,
                         (const bf16_t*)dy, offsets, p.n, (const bf16_t*)w2, (const bf16_t*)g, (const bf16_t*)u,
                         (bf16_t*)dgp, (bf16_t*)dup, p.d, p.f, ntn);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  WeightGrads w{};
  int nm = 0;
  auto want = [&](const void* P, const void* Q, void* C, int M, int N) {
    if (!C) return;
    w.m[nm++] = WeightGrad{(const bf16_t*)P, (const bf16_t*)Q, (bf16_t*)C, M, N};
  };
  want(h, dy, dw2, p.f, p.d);
  want(x, DG, dw1, p.d, p.f);
  want(x, DU, dw3, p.d, p.f);
  auto go = [&](auto mode) {
    return st_with_height(plan.input, [&](auto height) {
      constexpr int bn = InputCfg<height()>::BN;
      const int ntn = (p.d + bn - 1) / bn;
      InputGrad in{DG, DU, (const bf16_t*)w1, (const bf16_t*)w3, (bf16_t*)dx, p.d, p.f, ntn};
      unsigned gi = dx ? st_row_grid(p.rows_max, p.n, height(), ntn).x : 0, gw = nm ? st_grid(plan.units) : 0;
      if (plan.apart) {
        hipLaunchKernelGGL((input_weight_grad_bf16<height(), mode()>), dim3(gi), dim3(ST_NT), 0, st, in, w, 0, plan.div,
                           offsets, p.n);
        if (hipError_t e1 = hipGetLastError(); e1 != hipSuccess) return e1;
        in.dx = nullptr;
        gi = 0;
      }
      hipLaunchKernelGGL((input_weight_grad_bf16<height(), mode()>), dim3(std::min(gi + gw, st_grid(INT32_MAX))),
                         dim3(ST_NT), 0, st, in, w, nm, plan.div, offsets, p.n);
      return hipGetLastError();
    });
  };
  if (plan.mode == WG_SPLIT) {
    const int parts = plan.div;
    WeightSums sums{};
    char* at = dup + pad256((size_t)p.rows_max * p.f * p.elem());
    const int64_t count = (int64_t)p.n * p.d * p.f;
    for (int k = 0; k < nm; ++k, at += pad256((size_t)parts * count * 4)) {
      sums.part[k] = (const float*)at;
      sums.C[k] = w.m[k].C;
      w.m[k].C = (bf16_t*)at;
    }
    if ((e = go(std::integral_constant<int, WG_SPLIT>{})) != hipSuccess) return e;
    const int64_t blocks = (count / 8 + 255) / 256;
    hipLaunchKernelGGL(weight_grad_sum, dim3((unsigned)std::min<int64_t>(blocks, 2048), nm), dim3(256), 0, st, sums,
                       parts, count);
    return hipGetLastError();
  }
  if (plan.mode == WG_SHORT) return go(std::integral_constant<int, WG_SHORT>{});
  return go(std::integral_constant<int, WG_LONG>{});
}

}  // namespace moe
