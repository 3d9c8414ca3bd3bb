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
  // a group's scales (512 bytes) and zero points (256, gated: 256 of each matrix, half of them used)
  static constexpr int ZROW = GATED ? 512 : 256, ZOFF = SOFF + GPB * 512;
  static constexpr int SLOT = ZOFF + (ZERO ? GPB * ZROW : 0);
  static constexpr int NS = WM == 1 ? 4 : 3;                     // slots
  // copies of a wave per stage: rows, packed blocks, and pieces of 256 bytes of scales and
  // zero points dealt out over the waves (some twice, so that every wave issues as many)
  static constexpr int SP = 2 * GPB, PIECES = SP + (ZERO ? (GATED ? 2 : 1) * GPB : 0);
  static constexpr int CS = (PIECES + 7) / 8, COPIES = 2 * WM + 2 + CS;
  static constexpr int STORES = MT * (F32OUT ? NH : (NH + 1) / 2);
  typedef StOp<ST_ROWS, BM> X;
};

template <class C>
struct W4Ctx {
  typename C::X x;
  const char* w[2];        // packed runs of this wave's two blocks
  const char* s[C::CS];    // this wave's pieces of scales or zero points of the first stage
  uint32_t ssize[C::CS];   // bytes from there to the end of the matrix's, 0 for zero points that it has not
  uint32_t sstep[C::CS];   // bytes between stages
  uint32_t sdst[C::CS];    // where in a slot
  int nst;
};

// As bd_copy16, 4 bytes per lane.
__device__ __forceinline__ void bd_copy4(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t voff, uint32_t soff) {
  uint32_t keep;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
      "buffer_load_dword %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(keep)
      : "s"(lds), "v"(voff), "s"(r), "s"(soff)
      : "memory");
}

// A 256-byte piece of a stage's scales or zero points: group u, matrix or half of the columns hm.
struct W4Piece {
  int u, hm, dst;
  bool zero;
};
template <class C>
__device__ __forceinline__ W4Piece w4_piece(int at) {
  at %= C::PIECES;
  W4Piece q;
  q.zero = at >= C::SP;
  if (q.zero) at -= C::SP;
  q.u = __builtin_amdgcn_readfirstlane(at % C::GPB);
  q.hm = __builtin_amdgcn_readfirstlane(at / C::GPB);
  q.dst = q.zero ? C::ZOFF + C::ZROW * q.u + 256 * q.hm : C::SOFF + 512 * q.u + 256 * q.hm;
  return q;
}

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
    bd_copy4(gc_rsrc(c.s[v], c.ssize[v]), slot + c.sdst[v], 4u * (uint32_t)lane, (uint32_t)st * c.sstep[v]);
  }
}

// What a wave holds while it goes through its column tiles.  The group whose products
// are complete is scaled and added ("flushed") between the products of the next one, so
// that neither the matrix cores nor the vector unit waits for the other.
template <class C>
struct W4Wave {
  static constexpr int MT = C::MT, NT = C::NT, NH = C::NH, GPB = C::GPB, SPG = 4 / GPB;
  // Without zero points and with one group a stage, products start at -24 X instead of 0.
  static constexpr bool INIT = !C::ZERO && GPB == 1;
  int xo, wn;
  uint32_t mask, bits;     // of w4_unpack
  u32x4 x[MT][4];          // rows of the stage
  typename std::conditional<INIT, f32x4, float>::type X[MT][GPB];   // their group sums (INIT: times -24)
  f32x4 part[2][MT];       // products of a group, and of the one before
  u32x4 w, f;              // packed words of the tile, operand of the next k-step
  // the group to flush: scales, zero points, sums
  u32x2 sc;
  uint32_t zp;
  float z0, Xp[MT];

  __device__ __forceinline__ void clear() {
    sc = u32x2{0u, 0u};
    zp = 0;
    z0 = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      Xp[mt] = 0.f;
      part[1][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  __device__ __forceinline__ void read_x(const char* slot, int q) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) x[mt][q] = st_frag<ST_ROWS>(slot + (q >> 1) * C::XH, xo, q & 1, mt);
  }
  static constexpr int tile_of(int t, int& m) {
    m = C::GATED ? t / NH : 0;
    return C::GATED ? t % NH : t;
  }
  __device__ __forceinline__ u32x4 read_w(const char* slot, int t) const {
    int m = 0;
    const int at = NH * wn + tile_of(t, m);
    return *reinterpret_cast<const u32x4*>(slot + C::WOFF + 1024 * (at + 8 * m) + 16 * (threadIdx.x & 63));
  }
  __device__ __forceinline__ f32x4 start(int mt, int u) const {
    if constexpr (INIT) return X[mt][u];
    else return f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // Elements [k0, k1) of MT of the pending group's row tiles, products in part[b].
  __device__ __forceinline__ void flush(float (&acc)[MT][NT][4], int b, int t, int k0, int k1) {
    const float s[4] = {bf16_lo(sc[0]), bf16_hi(sc[0]), bf16_lo(sc[1]), bf16_hi(sc[1])};
#pragma unroll
    for (int mt = k0; mt < k1; ++mt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float z = C::ZERO ? z0 - (float)((zp >> (8 * r)) & 255u) : -24.f;
        const float v = INIT ? part[b][mt][r] : fmaf(z, Xp[mt], part[b][mt][r]);
        acc[mt][t][r] = fmaf(s[r], v, acc[mt][t][r]);
      }
  }
  // The group sums, and the last flush of the stage before.
  __device__ __forceinline__ void sums(float (&acc)[MT][NT][4]) {
    const uint32_t one = INIT ? 0xC1C0C1C0u : 0x3F803F80u;
    const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{one, one, one, one});
#pragma unroll
    for (int u = 0; u < GPB; ++u) {
      f32x4 v[MT];
#pragma unroll
      for (int q = u * SPG; q < (u + 1) * SPG; ++q)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          v[mt] = mfma16(ones, __builtin_bit_cast(bf16x8, x[mt][q]), q == u * SPG ? f32x4{0.f, 0.f, 0.f, 0.f} : v[mt]);
      flush(acc, 1, NT - 1, u * MT / GPB, (u + 1) * MT / GPB);
#pragma unroll
      for (int k = 0; k < MT * SPG; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        if constexpr (INIT) X[mt][u] = v[mt];
        else X[mt][u] = v[mt][0];
    }
  }
  // Tile t of the stage; NEXT: the following stage's rows are read once they are no longer needed.
  template <bool NEXT>
  __device__ __forceinline__ void tile(const W4Args& p, const char* slot, const char* next, int t, float (&acc)[MT][NT][4]) {
    int m = 0;
    const int at = NH * wn + tile_of(t, m);
    const int col = C::COLS * m + 16 * at + 4 * ((threadIdx.x & 63) >> 4);
    u32x4 wn4 = w;
    if (t + 1 < NT) wn4 = read_w(slot, t + 1);
#pragma unroll
    for (int u = 0; u < GPB; ++u) {
      constexpr int total = NT * GPB;
      const int b = (t * GPB + u) & 1;
      static_assert(total % 2 == 0, "the parts alternate across stages");
      const u32x2 nsc = *reinterpret_cast<const u32x2*>(slot + C::SOFF + u * 512 + 2 * col);
      const uint32_t nzp =
          C::ZERO ? *reinterpret_cast<const uint32_t*>(slot + C::ZOFF + u * C::ZROW + col + (C::GATED ? 128 * m : 0)) : 0u;
      const int before = u ? t : t - 1;   // the tile to flush (t = 0, u = 0: done by sums)
#pragma unroll
      for (int j = 0; j < SPG; ++j) {
        const int q = u * SPG + j;
        const u32x4 now = f;
        if (q < 3) f = w4_unpack(w[q + 1], mask, bits);
        else if (t + 1 < NT) f = w4_unpack(wn4[0], mask, bits);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          part[b][mt] = st_mfma(now, x[mt][q], j ? part[b][mt] : start(mt, u));
        if (before >= 0) flush(acc, b ^ 1, before, j * MT / SPG, (j + 1) * MT / SPG);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, C::ZERO ? 5 : 3, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (NEXT) read_x(next, q);   // into the registers just used
      }
      sc = nsc;
      zp = nzp;
      // a matrix without zero points reads zeros
      z0 = !C::ZERO ? -24.f : !C::GATED || (m ? p.z3 : p.z1) ? -16.f : -24.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        if constexpr (!INIT) Xp[mt] = X[mt][u];
    }
    w = wn4;
  }
  __device__ __forceinline__ void first_tiles(const W4Args& p, const char* slot, float (&acc)[MT][NT][4]) {
    w = read_w(slot, 0);
    sums(acc);
    f = w4_unpack(w[0], mask, bits);
#pragma unroll
    for (int t = 0; t + 1 < NT; ++t) tile<false>(p, slot, slot, t, acc);
  }
  __device__ __forceinline__ void last_tile(const W4Args& p, const char* slot, const char* next, float (&acc)[MT][NT][4]) {
    tile<true>(p, slot, next, NT - 1, acc);
  }
  __device__ __forceinline__ void flush_pending(float (&acc)[MT][NT][4]) { flush(acc, 1, NT - 1, 0, MT); }
};

template <class C>
__global__ __launch_bounds__(ST_NT, 1) void w4_tile(W4Args p, int ntn) {
  __shared__ __attribute__((aligned(16))) char ring[C::NS * C::SLOT];
  constexpr int MT = C::MT, NT = C::NT, NH = C::NH, GPB = C::GPB;
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
      const W4Piece q = w4_piece<C>(wave + 8 * v);
      const bool m = C::GATED && q.hm;
      const uint8_t* zp = m ? p.z3 : p.z1;
      const uint32_t row = (uint32_t)p.N * (q.zero ? 1u : 2u);   // bytes of a group
      const uint32_t skip = row * (uint32_t)q.u + (C::GATED || q.zero ? 0u : 256u * (uint32_t)q.hm);
      const uint32_t size = q.zero && !zp ? 0u : (uint32_t)p.groups * row;
      const char* from = (q.zero ? (const char*)(zp + go) : (const char*)((m ? p.s3 : p.s1) + go)) + skip;
      const uint64_t at = reinterpret_cast<uint64_t>(from);   // scalar: descriptors are made of it
      c.s[v] = reinterpret_cast<const char*>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at) |
                                             (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) << 32);
      c.ssize[v] = __builtin_amdgcn_readfirstlane(size > skip ? size - skip : 0u);
      c.sstep[v] = __builtin_amdgcn_readfirstlane(row * (uint32_t)GPB);
      c.sdst[v] = __builtin_amdgcn_readfirstlane(q.dst);
    }
    return t;
  };
  auto prologue = [&]() {
    // what setup loaded is here: else the compiler waits for it inside the loop over the
    // stages, and there for every copy as well
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
#pragma unroll
    for (int s = 0; s < C::NS - 1; ++s) w4_issue(p, c, lbase + s * C::SLOT, s);
  };
  StTile tile = setup(L);
  prologue();
  bool stores = false;
  for (;;) {
    float acc[MT][NT][4];   // single values: as vectors they are moved about at every branch
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[mt][t][r] = 0.f;
    // the first stage; newer are the other stages of the prologue and the stores of the tile before
    if (stores) st_sync<(C::NS - 2) * C::COPIES + C::STORES>();
    else st_sync<(C::NS - 2) * C::COPIES>();
    W4Wave<C> v;
    v.xo = xo;
    v.wn = wn;
    v.mask = w4_mask();
    v.bits = w4_bits();
    v.clear();
#pragma unroll
    for (int q = 0; q < 4; ++q) v.read_x(ring, q);
    uint32_t so = 0;   // slot offset of stage s
    for (int s = 0; s < c.nst; ++s) {
      v.first_tiles(p, ring + so, acc);
      // the next stage has arrived in every wave, and all are done with the one before;
      // stages past the last read zeros, so that the loop has no branches
      st_sync<(C::NS - 3) * C::COPIES>();
      w4_issue(p, c, lbase + (so == 0 ? (C::NS - 1) * C::SLOT : so - C::SLOT), s + C::NS - 1);
      const uint32_t to = so == (C::NS - 1) * C::SLOT ? 0 : so + C::SLOT;
      v.last_tile(p, ring + so, ring + to, acc);
      so = to;
    }
    v.flush_pending(acc);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");   // every wave is done with the ring
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
