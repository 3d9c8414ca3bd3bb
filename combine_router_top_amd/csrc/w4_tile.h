// Tiles of the 4-bit products (gfx950): 64 WM rows x 256 columns (gated: 128 of each
// matrix), 8 waves in a WM x (8 / WM) grid, each 64 rows by 16 NT columns, in stages of
// 128 K.
//
// The rows of a stage (two halves of 64 K in the ST_ROWS layout of seg_tile.h), its
// packed blocks and its scales are copied from memory straight into a ring of LDS slots.
// A wave holds its rows' fragments of a whole stage in registers and goes through its
// column tiles one by one: a tile's packed words become MFMA operands in registers (8
// values in 7 instructions, shared by the wave's four row tiles), a group's sums are
// scaled and added to the accumulators in fp32.  The group sums of the rows, which the
// offset of the operands needs, are a product with ones.
#pragma once

#include "w4.h"

namespace moe {

template <int WM_, int GPB_, bool ZERO_, bool GATED_, bool F32OUT_>
struct W4Cfg {
  static constexpr int WM = WM_, WN = 8 / WM, GPB = GPB_, MT = 4, BM = 64 * WM;
  static constexpr bool ZERO = ZERO_, GATED = GATED_, F32OUT = F32OUT_;
  static constexpr int NT = 16 / WN, NH = GATED ? NT / 2 : NT;   // a wave's weight and output tiles
  static constexpr int COLS = GATED ? 128 : 256;                 // output columns of a tile
  static constexpr int XH = BM * 128;                            // bytes of half a stage's rows
  static constexpr int WOFF = 2 * XH, SOFF = WOFF + 16 * 1024;   // packed blocks, then scales, zero points
  static constexpr int SROW = 512, ZROW = 256;                   // bytes of a group's scales, zero points (256 columns)
  static constexpr int ZOFF = SOFF + GPB * SROW;
  static constexpr int SLOT = ZOFF + (ZERO ? GPB * ZROW : 0);
  static constexpr int NS = WM == 1 ? 4 : 3;                     // slots
  // copies of a wave per stage: rows, packed blocks, and rows of scales and zero points
  // dealt out over the waves (some twice, so that every wave issues as many)
  static constexpr int PIECES = (GATED ? 2 : 1) * GPB * (ZERO ? 2 : 1);
  static constexpr int CS = (PIECES + 7) / 8, COPIES = 2 * WM + 2 + CS;
  static constexpr int STORES = MT * (F32OUT ? NH : (NH + 1) / 2);
  typedef StOp<ST_ROWS, BM> X;
};

template <class C>
struct W4Ctx {
  typename C::X x;
  const char* w[2];        // packed runs of this wave's two blocks
  const char* s[C::CS];    // this wave's pieces of scales or zero points, from the matrix's first group
  int nst;
};

// The copies of stage st into the slot at LDS address `slot`.
template <class C>
__device__ __forceinline__ void w4_issue(const W4Args& p, const W4Ctx<C>& c, uint32_t slot, int st) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  st_issue(c.x, slot, 2 * st);
  st_issue(c.x, slot + C::XH, 2 * st + 1);
  const uint32_t run = (uint32_t)p.kb * 1024u;
#pragma unroll
  for (int v = 0; v < 2; ++v)
    bd_copy16(gc_rsrc(c.w[v], run), slot + C::WOFF + 1024 * (wave + 8 * v), 16u * (uint32_t)lane, (uint32_t)st * 1024u);
#pragma unroll
  for (int v = 0; v < C::CS; ++v) {
    // piece: [zero points][matrix][group]
    const int piece = (wave + 8 * v) % C::PIECES, u = piece % C::GPB, m = piece / C::GPB % (C::GATED ? 2 : 1);
    const bool z = C::ZERO && piece >= C::PIECES / 2;
    const uint32_t es = z ? 1u : 2u, cols = C::COLS;
    const uint32_t row = (uint32_t)(st * C::GPB + u) * (uint32_t)p.N * es, size = c.s[v] ? (uint32_t)p.groups * (uint32_t)p.N * es : 0u;
    // the lanes of one piece's columns
    if ((uint32_t)lane * 16u < cols * es)
      bd_copy16(gc_rsrc(c.s[v], size), slot + (z ? C::ZOFF + u * C::ZROW : C::SOFF + u * C::SROW) + m * cols * es,
                16u * (uint32_t)lane, row);
  }
}

template <class C>
__global__ __launch_bounds__(ST_NT, 1) void w4_tile(W4Args p, int ntn) {
  __shared__ __attribute__((aligned(16))) char ring[C::NS * C::SLOT];
  constexpr int MT = C::MT, NT = C::NT, NH = C::NH, GPB = C::GPB, SPG = 4 / GPB;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int total = (p.offsets ? st_row_blocks(p.offsets, p.n, C::BM, p.lo) : (p.M + C::BM - 1) / C::BM) * ntn;
  int L = st_first_tile();
  if (L >= total) return;
  const uint32_t lbase = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(dt_lds_t*)ring);
  const uint32_t run = (uint32_t)p.kb * 1024u;
  const int xo = st_lane<ST_ROWS>(MT * wm);
  W4Ctx<C> c;
  c.nst = p.kb;
  auto setup = [&](int at) {
    const StTile t = p.offsets ? st_tile_at(at, p.offsets, p.n, ntn, C::BM, p.lo)
                               : st_tile_of(at, 0, p.M, (p.M + C::BM - 1) / C::BM, ntn, C::BM);
    st_rows(c.x, p.a + (int64_t)t.r0 * p.K, (uint32_t)p.K * 2, t.R, (uint32_t)p.K * 2);
    const int64_t eo = (int64_t)t.e * p.ntiles;
#pragma unroll
    for (int v = 0; v < 2; ++v) {   // packed blocks wave and wave + 8 (gated: the second matrix)
      const int tile = C::COLS / 16 * t.nt + (C::GATED ? wave : wave + 8 * v);
      c.w[v] = (C::GATED && v ? p.b3 : p.b1) + (eo + min(tile, p.ntiles - 1)) * run;
    }
    const int64_t go = (int64_t)t.e * p.groups * p.N + C::COLS * t.nt;
#pragma unroll
    for (int v = 0; v < C::CS; ++v) {
      const int piece = (wave + 8 * v) % C::PIECES, m = piece / GPB % (C::GATED ? 2 : 1);
      const bool z = C::ZERO && piece >= C::PIECES / 2;
      const uint8_t* zp = m ? p.z3 : p.z1;
      c.s[v] = z ? (zp ? (const char*)(zp + go) : nullptr) : (const char*)((m ? p.s3 : p.s1) + go);
    }
    return t;
  };
  auto prologue = [&]() {
#pragma unroll
    for (int s = 0; s < C::NS - 1; ++s)
      if (s < c.nst) w4_issue(p, c, lbase + s * C::SLOT, s);
  };
  StTile tile = setup(L);
  prologue();
  bool stores = false;
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
  for (;;) {
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[mt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint32_t so = 0;   // slot offset of stage s
    for (int s = 0; s < c.nst; ++s) {
      // this stage has arrived in every wave, and all are done with the one before
      if (s == 0 && stores) {
        const int later = min(C::NS - 2, c.nst - 1);
        if (later == 2) st_sync<2 * C::COPIES + C::STORES>();
        else if (later == 1) st_sync<C::COPIES + C::STORES>();
        else st_sync<C::STORES>();
      } else {
        st_sync_n<C::COPIES>(min(C::NS - 2, c.nst - 1 - s));
      }
      const uint32_t free = so == 0 ? (C::NS - 1) * C::SLOT : so - C::SLOT;
      if (s + C::NS - 1 < c.nst) w4_issue(p, c, lbase + free, s + C::NS - 1);
      const char* slot = ring + so;
      u32x4 x[MT][4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) x[mt][q] = st_frag<ST_ROWS>(slot + (q >> 1) * C::XH, xo, q & 1, mt);
      float X[MT][GPB];
#pragma unroll
      for (int u = 0; u < GPB; ++u)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = u * SPG; q < (u + 1) * SPG; ++q) v = mfma16(ones, __builtin_bit_cast(bf16x8, x[mt][q]), v);
          X[mt][u] = v[0];
        }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int h = C::GATED ? t % NH : t, m = C::GATED ? t / NH : 0;
        const int at = NH * wn + h;   // of the matrix's tiles in this block
        const u32x4 w = *reinterpret_cast<const u32x4*>(slot + C::WOFF + 1024 * (at + 8 * m) + 16 * lane);
#pragma unroll
        for (int u = 0; u < GPB; ++u) {
          f32x4 part[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) part[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = u * SPG; q < (u + 1) * SPG; ++q) {
            const u32x4 f = w4_unpack(w[q]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) part[mt] = st_mfma(f, x[mt][q], part[mt]);
          }
          const int col = C::COLS * m + 16 * at + 4 * g;
          const u32x2 s2 = *reinterpret_cast<const u32x2*>(slot + C::SOFF + u * C::SROW + 2 * col);
          const float sc[4] = {bf16_lo(s2[0]), bf16_hi(s2[0]), bf16_lo(s2[1]), bf16_hi(s2[1])};
          // a matrix without zero points reads zeros here
          const float z0 = C::ZERO && (m ? p.z3 : p.z1) ? -16.f : -24.f;
          const uint32_t zp = C::ZERO ? *reinterpret_cast<const uint32_t*>(slot + C::ZOFF + u * C::ZROW + col) : 0u;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float z = C::ZERO ? z0 - (float)((zp >> (8 * r)) & 255u) : z0;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              acc[mt][t][r] = fmaf(sc[r], fmaf(z, X[mt][u], part[mt][r]), acc[mt][t][r]);
          }
        }
      }
      so = so == (C::NS - 1) * C::SLOT ? 0 : so + C::SLOT;
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // every wave is done with the ring
    const int next = L + (int)gridDim.x;
    const StTile done = tile;
    if (next < total) {
      tile = setup(next);
      prologue();
    }
    __builtin_amdgcn_sched_barrier(0);
    constexpr int ES = C::F32OUT ? 4 : 2;
    const StOut out = st_out((char*)p.c + (int64_t)done.r0 * p.N * ES, (int64_t)p.N * ES, done.R);
    const int col0 = C::COLS * done.nt + 16 * NH * wn;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int row = 64 * wm + 16 * mt + i;
      f32x4 v[NH];
#pragma unroll
      for (int t = 0; t < NH; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[t][r] = C::GATED ? silu_mul(acc[mt][t][r], acc[mt][t + NT - NH][r]) : acc[mt][t][r];
      if constexpr (C::F32OUT) {
#pragma unroll
        for (int t = 0; t < NH; ++t) {
          const int at = col0 + 16 * t + 4 * g;
          st_put(out, row, 4u * (uint32_t)at, at < p.N, __builtin_bit_cast(u32x4, v[t]));
        }
      } else if constexpr (NH == 1) {   // 4 columns a lane
        const int at = col0 + 4 * g;
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{cvt_bf16x2(v[0][0], v[0][1]), cvt_bf16x2(v[0][2], v[0][3])}, out.r,
                                              at < p.N ? (uint32_t)row * out.ld + 2u * (uint32_t)at : 0xFFFFFFF0u, 0, 0);
      } else {
#pragma unroll
        for (int t = 0; t < NH; t += 2) {
          const int at = col0 + 16 * t + 8 * g;
          st_put(out, row, 2u * (uint32_t)at, at < p.N, st_pack8(v[t], v[t + 1]));
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    if (next >= total) return;
    L = next;
    stores = true;
  }
}

template <bool GATED, bool F32OUT, int WM, int GPB, bool ZERO>
static hipError_t launch_w4_tile(const W4Args& p, int64_t rows_max, hipStream_t st) {
  using C = W4Cfg<WM, GPB, ZERO, GATED, F32OUT>;
  const int ntn = (p.N + C::COLS - 1) / C::COLS;
  hipLaunchKernelGGL(w4_tile<C>, st_row_grid(rows_max, p.n, WM, ntn), dim3(ST_NT), 0, st, p, ntn);
  return hipGetLastError();
}

template <bool GATED, bool F32OUT>
static hipError_t launch_w4_tiles(const W4Args& p, int group, int height, int64_t rows_max, hipStream_t st) {
  const bool zero = p.z1 || (GATED && p.z3);
  auto with = [&](auto gpb, auto z) {
    return height == 1 ? launch_w4_tile<GATED, F32OUT, 1, gpb(), z()>(p, rows_max, st)
                       : launch_w4_tile<GATED, F32OUT, 2, gpb(), z()>(p, rows_max, st);
  };
  auto grouped = [&](auto gpb) {
    return zero ? with(gpb, std::true_type{}) : with(gpb, std::false_type{});
  };
  return group == 32   ? grouped(std::integral_constant<int, 4>{})
         : group == 64 ? grouped(std::integral_constant<int, 2>{})
                       : grouped(std::integral_constant<int, 1>{});
}

}  // namespace moe
