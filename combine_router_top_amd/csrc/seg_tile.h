// Tiles of a product over expert segments whose two operands may lie in memory
// in any of three ways (gfx950): the products of the experts' training forward
// and backward passes (bf16) and of the 8-bit experts (int8) share this core.
//
// A workgroup of 8 waves computes (64 MT) x 256 tiles, MT = 2, 3 or 4, or, for
// small problems, 64 x 128 tiles, in stages of 128 bytes of K (64 bf16 or 128
// int8 values, two 16x16 MFMA k-steps).  Wave (wm, wn) = (w & 3, w >> 2)
// multiplies 16 MT tile rows by half of the tile's columns.  Both operands of a
// stage are copied from memory straight into LDS (16 bytes per lane and
// instruction), the rows into a ring of NA slots and the columns into one of NB.
// While a wave multiplies one k-step from registers it reads the fragments of
// the next.  A stage costs one barrier, in
// its middle: by then every wave holds the stage's second half in registers,
// so its slots may be refilled, and the wait before it has seen the next
// stage's copies arrive.
//
// Why stages of 128 bytes: an operand whose rows are contiguous along K is read
// in pieces of one stage, and the address unit of a compute unit spends about
// 44 cycles on an instruction of sixteen 64-byte pieces against 22 on one of
// eight 128-byte pieces (whole cache lines, half the requests to L2).  With
// 64-byte stages that unit was busy 77% of the time and bounded the kernel.
//
// Operand layouts in memory and in a slot (W tile rows or columns):
//   ST_ROWS   row r of the operand is contiguous along K: 128-byte rows, 16-byte
//             piece q kept at q ^ ((r >> 1) & 7), so that every pass of a
//             fragment read (8 rows of one piece and 8 of its neighbour, see
//             dma_tile.h) meets 16 distinct bank groups.
//   ST_PANEL  row-major [K][ld], the operand's index contiguous (the products
//             that sum over a segment's rows): half-panels of 64 K-rows x 128
//             columns, piece q of row j kept at q ^ 2 sigma(j) as in dma_big.h;
//             a fragment is two transposing 8-byte reads.  bf16 only.
//   ST_PACK   int8 weights in MFMA operand order, 1 KB per 16 columns x 64 K:
//             copied and read linearly, without bank conflicts.
//
// The MFMA takes the column operand first, so a product lane holds 4
// consecutive columns of one row: lane (i, g) = (l % 16, l / 16) of wave
// (wm, wn) holds in acc[mt][t] row 16 MT wm + 16 mt + i, columns WN wn + 16 t
// + 4 g .. + 3 (WN: the columns of a wave).  st_swap_pair exchanges two column
// tiles between lane groups so that a lane holds 8 consecutive columns: 16-byte
// stores, whole 64-byte sectors per row.
//
// Workgroups are persistent (one per compute unit).  The first stages of the
// next tile are copied before the epilogue of this one, and its first waits
// count the epilogue's stores as outstanding (loads and stores retire in
// order), so that the stores of a tile drain while the next is loaded and
// multiplied.  An epilogue that loads itself (g and u of the gate gradient, the
// scales of the 8-bit tiles, a spilled register: keep_up_bf16<4>, keep_down_bf16<4>
// and the gated i8_tile<4> have 16 to 36 bytes of scratch a lane) waits for those first
// copies too, for the same reason.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "gemm_core.h"
#include "dma_tile.h"
#include "dma_big.h"
#include "kernels.h"
#include "tile_rules.h"

namespace moe {

enum { ST_ROWS = 0, ST_PANEL = 1, ST_PACK = 2 };

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int ST_NT = 512;     // threads

// One operand of W tile rows (or columns): state of its copies.
template <int L, int W>
struct StOp {
  static constexpr int C = W / 64;               // copies per wave per stage
  static constexpr int BYTES = W * ST_KB;        // bytes of a stage
  const char* base[L == ST_PACK ? C / 2 : 1];    // wave-uniform
  uint32_t v[L == ST_PANEL ? 2 : 1];             // lane source offsets at stage 0
  uint32_t ld;                                   // bytes between rows (ST_ROWS) or K-rows (ST_PANEL)
  uint32_t size;                                 // descriptor bytes (ST_ROWS, ST_PACK)
  uint32_t kbytes;                               // ST_ROWS: bytes of a row
  int krows;                                     // ST_PANEL: valid K-rows
};

// ST_ROWS: `rows` valid rows (>= 1) of `ld` bytes from base, kbytes (a multiple
// of 16) of each read.  Rows past the last valid one lie outside the descriptor
// and read zeros; so do the pieces of the last stage past a row's end, whose
// lanes are sent outside the descriptor.
template <int W>
__device__ __forceinline__ void st_rows(StOp<ST_ROWS, W>& o, const void* base, uint32_t ld, int rows,
                                        uint32_t kbytes) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // copy c of wave w: rows 64 c + 8 w .. + 7 (the swizzle does not depend on c)
  const int r = 8 * wave + (lane >> 3);
  o.base[0] = (const char*)base;
  o.v[0] = (uint32_t)r * ld + 16u * (uint32_t)((lane & 7) ^ ((r >> 1) & 7));
  o.ld = ld;
  o.size = (uint32_t)(min(rows, W) - 1) * ld + kbytes;
  o.kbytes = kbytes;
}

// ST_PANEL: K-rows [0, krows) of ld2 bytes from base, columns col0 .. col0 + W
// - 1 of which those below ncols are read; K-rows past krows read zeros.  With
// base2 the two half-panels are columns col0 .. col0 + 127 of two matrices.
template <int W>
__device__ __forceinline__ void st_panel(StOp<ST_PANEL, W>& o, const void* base, uint32_t ld2,
                                         int krows, int col0, int ncols, const void* base2 = nullptr) {
  static_assert(W == 256, "two half-panels");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // copy c of wave w: K-rows 16 (w % 4) + 4 c .. + 3 of half-panel w / 4;
  // sigma depends on c through c / 2
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int sig = ((lane >> 4) & 3) | (h << 2);
    const int col = col0 + (base2 ? 0 : 128 * (wave >> 2)) + 8 * ((lane & 15) ^ (2 * sig));
    const int j = 16 * (wave & 3) + 8 * h + (lane >> 4);
    o.v[h] = col < ncols ? (uint32_t)j * ld2 + 2u * (uint32_t)col : GC_OOR;
  }
  o.base[0] = (const char*)(base2 && (wave >> 2) ? base2 : base);
  o.ld = ld2;
  o.krows = krows;
  o.size = 0;
}

// ST_PACK: 16-column tiles nt0, nt0 + 1, .. of the packed matrix b1 of `ntiles`
// of them, each a run of `run` bytes (1 KB per 64 K); SPLIT: the first half of
// the columns from b1, the second, the same tiles, from b3.  Tiles past the last
// repeat it (their columns are never stored).
template <bool SPLIT, int W>
__device__ __forceinline__ void st_pack(StOp<ST_PACK, W>& o, const char* b1, const char* b3, int nt0, int ntiles,
                                        uint32_t run) {
  constexpr int H = W / 32;   // tiles of one half
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int c = 0; c < W / 128; ++c) {
    const int t = wave + 8 * c;
    const char* b = SPLIT && t >= H ? b3 : b1;
    o.base[c] = b + (int64_t)min(nt0 + (SPLIT && t >= H ? t - H : t), ntiles - 1) * run;
  }
  o.v[0] = 16u * (uint32_t)(threadIdx.x & 63);
  o.ld = 0;
  o.size = run;
}

// A wave-uniform quotient in a scalar register: the division runs on the vector
// unit, and what is derived from it (descriptors, offsets) has to be scalar.
__device__ __forceinline__ int st_div(int a, int b) { return __builtin_amdgcn_readfirstlane(a / b); }

// The copies of stage st of one operand into its slot at LDS address lds.
template <int L, int W>
__device__ __forceinline__ void st_issue(const StOp<L, W>& o, uint32_t lds, int st) {
  constexpr int C = StOp<L, W>::C;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (L == ST_ROWS) {
    const __amdgpu_buffer_rsrc_t r = gc_rsrc(o.base[0], o.size);
    const int lane = threadIdx.x & 63;
    const uint32_t piece = 16u * (uint32_t)((lane & 7) ^ (((8 * wave + (lane >> 3)) >> 1) & 7));
    const uint32_t v = (uint32_t)st * ST_KB + piece < o.kbytes ? o.v[0] : GC_OOR;
#pragma unroll
    for (int c = 0; c < C; ++c)
      bd_copy16(r, lds + 1024 * (wave + 8 * c), v, (uint32_t)st * ST_KB + (uint32_t)(64 * c) * o.ld);
  } else if constexpr (L == ST_PANEL) {
    // a descriptor per stage: a segment may span more than 32 bits
    // (the saturated row count is formed on the vector unit; the descriptor is scalar)
    const int rows = __builtin_amdgcn_readfirstlane(max(0, min(64, o.krows - 64 * st)));
    const __amdgpu_buffer_rsrc_t r = gc_rsrc(o.base[0] + (int64_t)st * 64 * o.ld, (uint32_t)rows * o.ld);
    const uint32_t at = lds + 16384 * (wave >> 2) + 4096 * (wave & 3);
#pragma unroll
    for (int c = 0; c < C; ++c)
      bd_copy16(r, at + 1024 * c, o.v[c >> 1], (uint32_t)(4 * (c & 1)) * o.ld);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
      bd_copy16(gc_rsrc(o.base[c >> 1], o.size), lds + 2048 * (wave + 8 * (c >> 1)) + 1024 * (c & 1), o.v[0],
                (uint32_t)st * 2048u + 1024u * (c & 1));
  }
}

// Lane offset, inside the operand's slot, of the fragment of a wave's first
// 16-wide tile t0 for k-step 0.
template <int L>
__device__ __forceinline__ int st_lane(int t0) {
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  if constexpr (L == ST_ROWS) return (16 * t0 + i) * ST_KB + 16 * (g ^ ((i >> 1) & 7));
  if constexpr (L == ST_PACK) return 2048 * t0 + 16 * lane;
  const int sig = (i >> 2) | ((g & 1) << 2);
  const int base = (8 * g + (i >> 2)) * BD_HPROW + 32 * sig + 8 * (i & 3);
  return (t0 >> 3) * 16384 + (base ^ (32 * (t0 & 7)));   // t0 & 7 = 0 or 4
}

// Fragment (16 bytes) of the wave's tile t and k-step ks.  ST_PANEL tiles of a
// wave lie in one half-panel and t0 is a multiple of the wave's tile count, so
// the tile index enters by XOR, as does the k-step of ST_ROWS.
template <int L>
__device__ __forceinline__ u32x4 st_frag(const char* slot, int lane_off, int ks, int t) {
  if constexpr (L == ST_PANEL) {
    const char* p = slot + (lane_off ^ (32 * (t & 7))) + 16384 * (t >> 3) + 8192 * ks;
    const s16x4 lo = dt_tr16(p), hi = dt_tr16(p + 4 * BD_HPROW);
    return __builtin_bit_cast(u32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  } else if constexpr (L == ST_ROWS) {
    return *reinterpret_cast<const u32x4*>(slot + (lane_off ^ (64 * ks)) + 2048 * t);
  } else {
    return *reinterpret_cast<const u32x4*>(slot + lane_off + 1024 * ks + 2048 * t);
  }
}

__device__ __forceinline__ f32x4 st_mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  return mfma16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c);
}
__device__ __forceinline__ i32x4 st_mfma(const u32x4& a, const u32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c,
                                               0, 0, 0);
}

// Tile configuration.  MT = 1: the small tile, 64 x 128 (64 x 256 for a gated pair
// of ST_PANEL matrices).  NP phases of operands follow one another along K (the
// input gradient sums two products); all have the same shape.  SPLIT: half of the
// columns are of one matrix, the others the same columns of a second (gate and up
// products of one h column meet in one lane: acc[mt][t] and acc[mt][t + NT / 2]).
// STORES: store instructions of a wave's epilogue, every one of them
// unconditional.  SHORT: two slots for each operand, for st_run_short.  ROT: K
// starts at stage ctx.rot and wraps around.
template <int MT_, int LA_, int LB_, typename AccT_, int NP_, bool SPLIT_, int STORES_, bool SHORT_ = false,
          int BN_ = MT_ == 1 ? 128 : 256, bool ROT_ = false>
struct StCfg {
  static constexpr int MT = MT_, LA = LA_, LB = LB_, NP = NP_, STORES = STORES_;
  static constexpr bool SPLIT = SPLIT_, ROT = ROT_;
  static constexpr int BM = 64 * MT, BN = BN_;
  static constexpr int NT = BN / 32, WN = BN / 2;              // a wave's column tiles and columns
  typedef AccT_ Acc[MT][NT];
  typedef StOp<LA, BM> A;
  typedef StOp<LB, BN> B;
  // slots: the columns (weights, from HBM) three deep where LDS allows; small
  // tiles, of which a compute unit may have one alone, as deep as LDS holds,
  // since nothing else hides the latency of their loads
  static constexpr int DEEP = BN == 128 ? 6 : 4;
  static constexpr int NA = MT == 1 ? DEEP : BM == 128 && !SHORT_ ? 3 : 2, NB = MT == 1 ? DEEP : SHORT_ ? 2 : 3;
  static constexpr int AREG = NA * A::BYTES;                   // the column slots follow the row slots
  static constexpr int LDS = AREG + NB * B::BYTES;             // 128 to 160 KB (all there is)
  static constexpr int CA = A::C, CB = B::C;                   // copies per wave per stage
  // copies issued after those of stage s + 1 when stage s reaches its middle
  static constexpr int LATER = (NB > NA ? CB : 0) + (NA - 2) * (CA + CB);
  static_assert(NB == NA || NB == NA + 1, "issue order");
};

template <class Cfg>
struct StCtx {
  typename Cfg::A a[Cfg::NP];
  typename Cfg::B b[Cfg::NP];
  int nst1;          // stages of a phase
  int nst;           // stages in all
  int rot;           // first stage (ROT)
};

template <class Cfg>
struct StFrag {
  u32x4 x[Cfg::MT], w[Cfg::NT];
};

// The copies of stage st into the slot at LDS address `at`.
template <class Cfg>
__device__ __forceinline__ void st_issue_a(const StCtx<Cfg>& c, uint32_t at, int st) {
  if (Cfg::ROT) {
    st += c.rot;
    if (st >= c.nst) st -= c.nst;
  }
  if (Cfg::NP > 1 && st >= c.nst1) st_issue(c.a[Cfg::NP - 1], at, st - c.nst1);
  else st_issue(c.a[0], at, st);
}
template <class Cfg>
__device__ __forceinline__ void st_issue_b(const StCtx<Cfg>& c, uint32_t at, int st) {
  if (Cfg::ROT) {
    st += c.rot;
    if (st >= c.nst) st -= c.nst;
  }
  if (Cfg::NP > 1 && st >= c.nst1) st_issue(c.b[Cfg::NP - 1], at, st - c.nst1);
  else st_issue(c.b[0], at, st);
}

// Wait until at most N of this wave's copies and stores are outstanding and its
// LDS reads have completed, then barrier.
template <int N>
__device__ __forceinline__ void st_sync() {
  bd_sync<(N < 63 ? N : 63)>();   // the counter's six bits; a smaller count waits for more
}

template <class Cfg>
struct StLane {
  int ao, bo;        // lane fragment offsets in a slot
  uint32_t lbase;    // LDS address of the ring
};

template <class Cfg>
__device__ __forceinline__ StLane<Cfg> st_lanes(char* ring) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  StLane<Cfg> l;
  l.lbase = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(dt_lds_t*)ring);
  l.ao = st_lane<Cfg::LA>(Cfg::MT * (wave & 3));
  l.bo = st_lane<Cfg::LB>((Cfg::SPLIT ? Cfg::NT / 2 : Cfg::NT) * (wave >> 2));
  return l;
}

// Where a wave's column tile t lies in a slot, from its first.
template <class Cfg>
__device__ __forceinline__ constexpr int st_slot_tile(int t) {
  constexpr int H = Cfg::NT / 2;
  return Cfg::SPLIT ? t % H + 2 * H * (t / H) : t;
}

// Multiply F; with READ, read k-step ks of stage st into G meanwhile, from the
// slots at as and bs.  Once a wave has its first products under way it takes
// priority over the other wave of its SIMD, which then waits, copies or reads
// LDS beside them instead of both multiplying in step (dense 8-expert backward
// pass 19.6 -> 18.7 ms, 4096 x 14336 x 4096 int8 product 241 -> 222 us; the
// order of reads and products inside a k-step is left to the compiler).
template <bool READ, class Cfg>
__device__ __forceinline__ void st_kstep(const StLane<Cfg>& l, const char* as, const char* bs, int ks,
                                         const StFrag<Cfg>& F, StFrag<Cfg>& G, typename Cfg::Acc& acc) {
  constexpr int MT = Cfg::MT;
  __builtin_amdgcn_sched_barrier(0);
  if (READ) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) G.x[mt] = st_frag<Cfg::LA>(as, l.ao, ks, mt);
  }
#pragma unroll
  for (int t = 0; t < Cfg::NT; ++t) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt][t] = st_mfma(F.w[t], F.x[mt], acc[mt][t]);
    if (t == 0) __builtin_amdgcn_s_setprio(1);
    if (READ) {
      G.w[t] = st_frag<Cfg::LB>(bs, l.bo, ks, st_slot_tile<Cfg>(t));
    }
  }
  __builtin_amdgcn_s_setprio(0);
  __builtin_amdgcn_sched_barrier(0);
}

template <class Cfg>
__device__ __forceinline__ void st_clear(typename Cfg::Acc& acc) {
#pragma unroll
  for (int a = 0; a < Cfg::MT; ++a)
#pragma unroll
    for (int t = 0; t < Cfg::NT; ++t) acc[a][t] = {};
}

// The copies of a tile's first stages, in the order A0 B0 A1 B1 (A2) (B2) ..
// Every wave must be done with the ring.
template <class Cfg>
__device__ __forceinline__ void st_prologue(const StCtx<Cfg>& c, const StLane<Cfg>& l) {
#pragma unroll
  for (int s = 0; s < Cfg::NB; ++s) {
    if (s < Cfg::NA && s < c.nst) st_issue_a(c, l.lbase + s * Cfg::A::BYTES, s);
    if (s < Cfg::NB && s < c.nst) st_issue_b(c, l.lbase + Cfg::AREG + s * Cfg::B::BYTES, s);
  }
}

// Wait until n (0 .. 5) newer stages of CNT copies may be outstanding.
template <int CNT>
__device__ __forceinline__ void st_sync_n(int n) {
  if (n >= 5) st_sync<5 * CNT>();
  else if (n == 4) st_sync<4 * CNT>();
  else if (n == 3) st_sync<3 * CNT>();
  else if (n == 2) st_sync<2 * CNT>();
  else if (n == 1) st_sync<CNT>();
  else st_sync<0>();
}

// Wait for stage s (0 or 1) of the prologue with S later stores outstanding.
// Small tiles wait for the stores as well: a workgroup has few of them.
template <int S, class Cfg>
__device__ __forceinline__ void st_wait_first(int s, int nst) {
  if constexpr (Cfg::MT == 1) {
    st_sync_n<Cfg::CA + Cfg::CB>(min(nst, Cfg::NA) - 1 - s);
    return;
  }
  constexpr int ST = Cfg::CA + Cfg::CB;                                       // a whole stage
  constexpr int THIRD = (Cfg::NA > 2 ? Cfg::CA : 0) + (Cfg::NB > 2 ? Cfg::CB : 0);
  if (s == 0) {
    if (nst >= 3) st_sync<ST + THIRD + S>();
    else if (nst == 2) st_sync<ST + S>();
    else st_sync<S>();
  } else {
    if (nst >= 3) st_sync<THIRD + S>();
    else st_sync<S>();
  }
}

// acc = the product over c.nst stages (>= 1) whose prologue has been issued,
// followed by `stores` (0 or Cfg::STORES) stores of the epilogue before.  At
// the end no copy is outstanding and every wave is done with the ring.
template <class Cfg>
__device__ __forceinline__ void st_accum(const StCtx<Cfg>& c, const StLane<Cfg>& l, const char* ring, bool stores,
                                         typename Cfg::Acc& acc) {
  st_clear<Cfg>(acc);
  if (stores) st_wait_first<Cfg::STORES, Cfg>(0, c.nst);
  else st_wait_first<0, Cfg>(0, c.nst);
  StFrag<Cfg> F, G;
#pragma unroll
  for (int mt = 0; mt < Cfg::MT; ++mt) F.x[mt] = st_frag<Cfg::LA>(ring, l.ao, 0, mt);
#pragma unroll
  for (int t = 0; t < Cfg::NT; ++t) F.w[t] = st_frag<Cfg::LB>(ring + Cfg::AREG, l.bo, 0, st_slot_tile<Cfg>(t));
  // slot offsets of stage s; stage s + NA (NB) takes the slot of stage s
  uint32_t as = 0, bs = Cfg::AREG;
  int s = 0;
  for (; s + 1 < c.nst; ++s) {
    st_kstep<true>(l, ring + as, ring + bs, 1, F, G, acc);
    if (s == 0) {
      if (stores) st_wait_first<Cfg::STORES, Cfg>(1, c.nst);
      else st_wait_first<0, Cfg>(1, c.nst);
    } else if (Cfg::MT == 1) {
      // stages s + 2 .. s + NA - 1, those of them that exist
      st_sync_n<Cfg::CA + Cfg::CB>(min(c.nst - 2 - s, Cfg::NA - 2));
    } else if (s + 2 < c.nst) {
      st_sync<Cfg::LATER>();
    } else {
      st_sync<0>();
    }
    if (s + Cfg::NA < c.nst) st_issue_a(c, l.lbase + as, s + Cfg::NA);
    const uint32_t free_b = bs;
    if (Cfg::MT == 1 && s + Cfg::NB < c.nst) st_issue_b(c, l.lbase + free_b, s + Cfg::NB);
    as = as == (Cfg::NA - 1) * Cfg::A::BYTES ? 0 : as + Cfg::A::BYTES;
    bs = bs == Cfg::AREG + (Cfg::NB - 1) * Cfg::B::BYTES ? Cfg::AREG : bs + Cfg::B::BYTES;
    st_kstep<true>(l, ring + as, ring + bs, 0, G, F, acc);
    // half a stage after the rows' copies, which spreads the requests
    if (Cfg::MT != 1 && s + Cfg::NB < c.nst) st_issue_b(c, l.lbase + free_b, s + Cfg::NB);
  }
  st_kstep<true>(l, ring + as, ring + bs, 1, F, G, acc);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  st_kstep<false>(l, ring, ring, 0, G, F, acc);
}

// ---------------------------------------------------------------------------
// epilogues
// ---------------------------------------------------------------------------
// Column tiles t (x) and t + 1 (y) of one row tile, one word of 2 packed or 1
// plain column per lane and register: afterwards lane group g holds, in (x, y)
// order, what groups 2 (g % 2) and 2 (g % 2) + 1 held of tile t + g / 2.
__device__ __forceinline__ void st_swap_pair(uint32_t& x, uint32_t& y) {
  const auto a = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[1], false, false);
  x = b[0];
  y = b[1];
}
__device__ __forceinline__ void st_swap_pair(float& x, float& y) {
  uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  st_swap_pair(a, b);
  x = __uint_as_float(a);
  y = __uint_as_float(b);
}

// Values of column tiles t and t + 1 as bf16: 8 consecutive columns per lane,
// 16 t + 8 g .. + 7 (g the lane group).
__device__ __forceinline__ u32x4 st_pack8(const float (&x)[4], const float (&y)[4]) {
  uint32_t x0 = cvt_bf16x2(x[0], x[1]), x1 = cvt_bf16x2(x[2], x[3]);
  uint32_t y0 = cvt_bf16x2(y[0], y[1]), y1 = cvt_bf16x2(y[2], y[3]);
  st_swap_pair(x0, y0);
  st_swap_pair(x1, y1);
  return u32x4{x0, x1, y0, y1};
}
__device__ __forceinline__ u32x4 st_pack8(const f32x4& x, const f32x4& y) {
  const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {y[0], y[1], y[2], y[3]};
  return st_pack8(a, b);
}

// Output rows of a tile: stores outside its rows or columns leave the
// descriptor, so that every store is issued and none needs a branch.
struct StOut {
  __amdgpu_buffer_rsrc_t r;
  uint32_t ld;   // bytes per row
};
__device__ __forceinline__ StOut st_out(void* base, int64_t ld, int rows) {
  return StOut{gc_rsrc(base, (uint32_t)rows * (uint32_t)ld), (uint32_t)ld};
}
// 16 bytes at (row, byte column), or nothing where !ok.  NT: non-temporal.
template <bool NT = false>
__device__ __forceinline__ void st_put(const StOut& o, int row, uint32_t byte, bool ok, const u32x4& v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, o.r, ok ? (uint32_t)row * o.ld + byte : 0xFFFFFFF0u, 0, NT ? 2 : 0);
}

// bf16 rows of a finished tile: its columns from col0, those below N.
template <int MT, int NT>
__device__ __forceinline__ void st_store_tile(const StOut& o, const f32x4 (&acc)[MT][NT], int col0, int N) {
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int k = 0; k < NT / 2; ++k) {
      const int col = col0 + 16 * NT * (wave >> 2) + 32 * k + 8 * q;
      st_put(o, 16 * MT * (wave & 3) + 16 * mt + i, 2u * (uint32_t)col, col < N,
             st_pack8(acc[mt][2 * k], acc[mt][2 * k + 1]));
    }
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

// ---------------------------------------------------------------------------
// row blocks of expert segments
// ---------------------------------------------------------------------------
constexpr int ST_GM = 8;        // row blocks of one expert that run together

struct StTile {
  int e, r0, R, nt;   // expert, first row, valid rows, column block
};

// Row blocks of bm rows of all n segments (those of at most lo rows have none).
// Every wave computes it by itself.
__device__ __forceinline__ int st_row_blocks(const int32_t* __restrict__ offsets, int n, int bm, int lo = 0) {
  const int lane = threadIdx.x & 63;
  int x = 0;
  for (int j = lane; j < n; j += 64) {
    const int cnt = offsets[j + 1] - offsets[j];
    x += cnt > lo ? (cnt + bm - 1) / bm : 0;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
  return __builtin_amdgcn_readfirstlane(x);
}

// Tile `local` of one segment of `rows` rows from row o, `blocks` row blocks:
// groups of ST_GM row blocks run through the column blocks together, so that
// neighbouring tiles share weight columns and an expert's rows in an L2.
__device__ __forceinline__ StTile st_tile_of(int local, int o, int rows, int blocks, int ntn, int bm) {
  const int mg = st_div(local, ST_GM * ntn);
  const int rem = local - mg * ST_GM * ntn;
  const int gsz = min(ST_GM, blocks - mg * ST_GM);
  const int nt = st_div(rem, gsz);
  const int mb = mg * ST_GM + (rem - nt * gsz);
  return StTile{0, __builtin_amdgcn_readfirstlane(o + mb * bm),
                __builtin_amdgcn_readfirstlane(min(bm, rows - mb * bm)), __builtin_amdgcn_readfirstlane(nt)};
}

// Tile L of (row blocks) * ntn, expert by expert.  Every wave searches by
// itself (64 experts a step), which leaves all of LDS to the rings.
__device__ __forceinline__ StTile st_tile_at(int L, const int32_t* __restrict__ offsets, int n, int ntn, int bm,
                                             int lo = 0) {
  const int lane = threadIdx.x & 63;
  const int q = st_div(L, ntn);   // the row block, counted over all experts
  StTile t{0, 0, 0, 0};
  for (int j0 = 0, before = 0; j0 < n; j0 += 64) {
    const int j = j0 + lane;
    const int o = j < n ? offsets[j] : 0;
    const int cnt = j < n ? offsets[j + 1] - o : 0;
    const int nrb = cnt > lo ? (cnt + bm - 1) / bm : 0;
    int x = nrb;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    const uint64_t hit = __ballot(before + x > q);
    if (hit) {
      const int at = __ffsll((unsigned long long)hit) - 1;
      const int blocks = __shfl(nrb, at), first = before + __shfl(x, at) - blocks;
      const int o0 = __shfl(o, at), rows = __shfl(cnt, at);
      t = st_tile_of(L - first * ntn, o0, rows, blocks, ntn, bm);
      t.e = __builtin_amdgcn_readfirstlane(j0 + at);
      return t;
    }
    before += __shfl(x, 63);
  }
  return t;
}

// Walk of the G persistent workgroups (G a multiple of 8) over `total` tiles:
// in every round each XCD (workgroup id mod 8 on this part) takes one run of
// G / 8 consecutive tiles, so that neighbouring tiles share an L2, and tiles of
// unequal length (experts of unequal row counts) spread over all XCDs.
__device__ __forceinline__ int st_first_tile() {
  return (int)(blockIdx.x & 7) * (int)(gridDim.x >> 3) + (int)(blockIdx.x >> 3);
}

// First tile of a second walk in the same launch, after one over `before` tiles:
// the workgroups that the first walk's last round left without a tile come first.
__device__ __forceinline__ int st_second_tile(int before) {
  const int G = (int)gridDim.x;
  const int at = st_first_tile() - (before - st_div(before, G) * G);
  return at < 0 ? at + G : at;
}

// The persistent loop.  setup(L, ctx) describes tile L and returns what
// finish(tile, acc) needs to store it, with exactly Cfg::STORES stores per wave.
// setup may leave ctx.nst = 0 (a tile of zeros).  first: this workgroup's first tile.
template <class Cfg, class Setup, class Finish>
__device__ __forceinline__ void st_run(int total, char* ring, const Setup& setup, const Finish& finish,
                                       int first = st_first_tile()) {
  const StLane<Cfg> l = st_lanes<Cfg>(ring);
  int L = first;
  if (L >= total) return;
  StCtx<Cfg> c;
  auto tile = setup(L, c);
  st_prologue(c, l);
  bool stores = false;
  for (;;) {
    typename Cfg::Acc acc;
    if (c.nst > 0) st_accum(c, l, ring, stores, acc);
    else st_clear<Cfg>(acc);
    const int next = L + (int)gridDim.x;
    const bool more = next < total;
    const auto done = tile;
    if (more) {
      tile = setup(next, c);
      st_prologue(c, l);
    }
    __builtin_amdgcn_sched_barrier(0);
    finish(done, acc);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    if (!more) return;
    L = next;
    stores = true;
  }
}

// The persistent loop for tiles of few stages (segments of a few hundred rows,
// where a tile is mostly loading and storing).  A workgroup takes units: runs of
// row blocks of one block of columns.  Two things differ from st_run:
//   - the copies run ahead of the products across tiles and units: the stages
//     form one sequence, and as soon as a stage's slots are free the next but
//     one is copied, so that a tile's operands arrive while its predecessor is
//     multiplied and stored;
//   - a unit of two stages (up to 128 K-rows; one is padded to two with zeros)
//     copies its columns once: stages alternate between the two slots, so the
//     columns of stage s stay in theirs from tile to tile.
// unit(U) gives a Unit with nst (stages, 0 or >= 2) and tiles; cols(unit, ctx)
// and rows(unit, j, ctx) describe its operands for row block j; finish(unit, j,
// acc) stores with exactly Cfg::STORES stores per wave.  first: this workgroup's
// first unit.
template <class Cfg, class UnitOf, class Cols, class Rows, class Finish>
__device__ __forceinline__ void st_run_short(int total, char* ring, const UnitOf& unit, const Cols& cols,
                                             const Rows& rows, const Finish& finish, int first = st_first_tile()) {
  static_assert(Cfg::NA == 2 && Cfg::NB == 2 && Cfg::NP == 1, "two slots, one phase");
  constexpr int CA = Cfg::CA, S = Cfg::STORES;
  const StLane<Cfg> l = st_lanes<Cfg>(ring);
  const int G = (int)gridDim.x;
  if (first >= total) return;
  // the copies' place: unit Up, its row block jp, that block's next stage sp
  int Up = first - G, jp = 0, sp = 0;
  int ahead = 0;   // stages copied or on their way, not yet multiplied
  StCtx<Cfg> p;
  auto up = unit(first);
  up.tiles = 0;   // before the first unit
  auto copy_next = [&](int slot) __attribute__((always_inline)) {
    while (up.nst == 0 || jp >= up.tiles) {
      Up += G;
      if (Up >= total) {
        Up = total;   // nothing left: stay here
        return;
      }
      up = unit(Up);
      jp = sp = 0;
      if (up.nst > 0) {
        cols(up, p);
        rows(up, 0, p);
      }
    }
    if (jp == 0 || up.nst > 2) st_issue_b(p, l.lbase + Cfg::AREG + slot * Cfg::B::BYTES, sp);
    st_issue_a(p, l.lbase + slot * Cfg::A::BYTES, sp);
    ++ahead;
    if (++sp == up.nst) {
      sp = 0;
      if (++jp < up.tiles) rows(up, jp, p);
    }
  };
  copy_next(0);
  copy_next(1);
  int slot = 0;
  bool stores = false;   // the last finish's stores may be outstanding
  for (int U = first; U < total; U += G) {
    const auto u = unit(U);
    for (int j = 0; j < u.tiles; ++j) {
      typename Cfg::Acc acc;
      st_clear<Cfg>(acc);
      if (u.nst > 0) {
        // this stage's copies; after them came the next stage's (at least its
        // rows) and the last tile's stores
        if (ahead > 1) {
          if (stores) st_sync<CA + S>();
          else st_sync<CA>();
        } else {
          if (stores) st_sync<S>();
          else st_sync<0>();
        }
        StFrag<Cfg> F, F1;
        const char* as = ring + slot * Cfg::A::BYTES;
        const char* bs = ring + Cfg::AREG + slot * Cfg::B::BYTES;
#pragma unroll
        for (int mt = 0; mt < Cfg::MT; ++mt) F.x[mt] = st_frag<Cfg::LA>(as, l.ao, 0, mt);
#pragma unroll
        for (int t = 0; t < Cfg::NT; ++t) F.w[t] = st_frag<Cfg::LB>(bs, l.bo, 0, t);
        int s = 0;
        for (; s + 1 < u.nst; ++s) {
          st_kstep<true>(l, ring + slot * Cfg::A::BYTES, ring + Cfg::AREG + slot * Cfg::B::BYTES, 1, F, F1, acc);
          // the next stage was copied before the stores only if this is the first
          if (s == 0 && stores) st_sync<S>();
          else st_sync<0>();
          --ahead;
          copy_next(slot);
          slot ^= 1;
          st_kstep<true>(l, ring + slot * Cfg::A::BYTES, ring + Cfg::AREG + slot * Cfg::B::BYTES, 0, F1, F, acc);
        }
        st_kstep<true>(l, ring + slot * Cfg::A::BYTES, ring + Cfg::AREG + slot * Cfg::B::BYTES, 1, F, F1, acc);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        --ahead;
        copy_next(slot);
        slot ^= 1;
        st_kstep<false>(l, ring, ring, 0, F1, F, acc);
      }
      __builtin_amdgcn_sched_barrier(0);
      finish(u, j, acc);
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      stores = true;
    }
  }
}

// ---------------------------------------------------------------------------
// host side: launches by tile height (tile_rules.h chooses it)
// ---------------------------------------------------------------------------
// Calls go with the height as a compile-time constant.
template <class Go>
inline hipError_t st_with_height(int h, const Go& go) {
  switch (h) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 3: return go(std::integral_constant<int, 3>{});
    default: return go(std::integral_constant<int, 4>{});
  }
}

// Grid over the row blocks that a batch can have at most.
inline dim3 st_row_grid(int64_t rows_max, int64_t n, int h, int ntn) {
  const int64_t blocks = std::min<int64_t>(rows_max / (64 * h) + std::min<int64_t>(n, rows_max), rows_max);
  return dim3(st_grid(blocks * ntn));
}

}  // namespace moe
