// Tiles of a product over expert segments whose two operands may lie in memory
// in any of three ways (gfx950): the products of the experts' backward pass
// (bf16) and of the 8-bit experts (int8) share this core.
//
// A workgroup of 8 waves computes a (64 MT) x 256 tile, MT = 2 or 4, in stages
// of 64 bytes of K (32 bf16 or 64 int8 values, one 16x16 MFMA k-step).  Wave
// (wm, wn) = (w & 3, w >> 2) multiplies 16 MT tile rows by 128 tile columns.
// Both operands of a stage are copied from memory straight into a slot of an
// LDS ring (16 bytes per lane and instruction); a wave holds the fragments of
// the stage it multiplies in registers, so all other slots are in flight or
// wait.  A stage is released by an explicit wait for the wave's own copies and
// one barrier, which also frees the slot that every wave has read.
//
// Operand layouts in memory and in a slot (W tile rows or columns):
//   ST_ROWS   row r of the operand is contiguous along K: 64-byte rows, 16-byte
//             piece q kept at q ^ dt_swa(r); a fragment is one 16-byte read.
//   ST_PANEL  row-major [K][ld], the operand's index contiguous (the products
//             that sum over a segment's rows): half-panels of 32 K-rows x 128
//             columns, piece q of row j kept at q ^ 2 sigma(j); a fragment is
//             two transposing 8-byte reads.  bf16 only.
//   ST_PACK   int8 weights in MFMA operand order, 1 KB per 16 columns x 64 K:
//             copied and read linearly, without bank conflicts.
// Both swizzles are those of dma_tile.h and dma_big.h, applied by the lane's
// choice of the source piece.
//
// The MFMA takes the column operand first, so a product lane holds 4
// consecutive columns of one row: lane (i, g) = (l % 16, l / 16) of wave
// (wm, wn) holds in acc[mt][t] row 16 MT wm + 16 mt + i, columns 128 wn + 16 t
// + 4 g .. + 3.
#pragma once

#include "common.h"
#include "gemm_core.h"
#include "dma_tile.h"
#include "dma_big.h"

namespace moe {

enum { ST_ROWS = 0, ST_PANEL = 1, ST_PACK = 2 };

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int ST_BN = 256;     // tile columns
constexpr int ST_KB = 64;      // bytes of K per stage
constexpr int ST_NT = 512;     // threads

// One operand of W tile rows (or columns): per-thread state of its copies.
template <int L, int W>
struct StOp {
  static_assert(W == 256 || W == 128, "tile sides of 128 or 256");
  static constexpr int C = W / 128;              // copies per wave per stage
  static constexpr int BYTES = W * ST_KB;        // bytes of a stage
  __amdgpu_buffer_rsrc_t r[L == ST_PACK ? C : 1];
  uint32_t v[L == ST_PANEL ? 1 : C];             // lane source offsets at stage 0
  uint32_t step;                                 // source bytes per stage
  uint32_t sub;                                  // ST_PANEL: bytes of 4 K-rows
  int dst;                                       // this wave's first destination in the region
};

// ST_ROWS: `rows` valid rows (>= 1) of `ld` bytes from base; K bytes per row.
// Rows past the last valid one repeat it.
template <int W>
__device__ __forceinline__ void st_rows(StOp<ST_ROWS, W>& o, const void* base, uint32_t ld, int rows,
                                        uint32_t kbytes) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  o.r[0] = gc_rsrc(base, (uint32_t)(min(rows, W) - 1) * ld + kbytes);
#pragma unroll
  for (int c = 0; c < W / 128; ++c) {
    const int r = 16 * (wave + 8 * c) + (lane >> 2);
    o.v[c] = (uint32_t)min(r, rows - 1) * ld + 16u * (uint32_t)((lane & 3) ^ dt_swa(r));
  }
  o.step = ST_KB;
  o.sub = 0;
  o.dst = 1024 * wave;
}

// ST_PANEL: K-rows [0, krows) of ld2 bytes from base, columns col0 .. col0 + W
// - 1 of which those below ncols are read; K-rows past krows read zeros (the
// descriptor ends there).  krows * ld2 < 2^32.
template <int W>
__device__ __forceinline__ void st_panel(StOp<ST_PANEL, W>& o, const void* base, uint32_t ld2,
                                         int krows, int col0, int ncols) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // W = 256: wave w copies K-rows 8 (w % 4) .. + 7 of half-panel w / 4 in two
  // copies; W = 128: K-rows 4 w .. + 3 of the one half-panel
  const int hp = W == 256 ? wave >> 2 : 0;
  const int j0 = W == 256 ? 8 * (wave & 3) : 4 * wave;
  const int j = j0 + (lane >> 4);
  const int sig = (j & 3) | (((j >> 3) & 1) << 2);
  const int col = col0 + 128 * hp + 8 * ((lane & 15) ^ (2 * sig));
  o.r[0] = gc_rsrc(base, (uint32_t)krows * ld2);
  o.v[0] = col < ncols ? (uint32_t)j * ld2 + 2u * (uint32_t)col : GC_OOR;
  o.step = 32 * ld2;
  o.sub = 4 * ld2;
  o.dst = hp * BD_HP + j0 * BD_HPROW;
}

// ST_PACK, one 128-column half c: 16-column tiles nt0 .. nt0 + 7 of a packed
// matrix of `ntiles` of them, each a run of `run` bytes (1 KB per 64 K); tiles
// past the last repeat it (their columns are never stored).
template <int W>
__device__ __forceinline__ void st_pack(StOp<ST_PACK, W>& o, int c, const void* base, int nt0, int ntiles,
                                        uint32_t run) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the descriptor starts at this wave's tile, so that its offsets stay below one run
  const int nt = min(nt0 + wave, ntiles - 1);
  o.r[c] = gc_rsrc((const char*)base + (int64_t)nt * run, run);
  o.v[c] = 16u * (uint32_t)lane;
  o.step = 1024;
  o.sub = 0;
  o.dst = 1024 * wave;
}

// The copies of stage st of one operand into its region at LDS address lds.
template <int L, int W>
__device__ __forceinline__ void st_issue(const StOp<L, W>& o, uint32_t lds, uint32_t st) {
  const uint32_t so = st * o.step;
#pragma unroll
  for (int c = 0; c < W / 128; ++c) {
    if constexpr (L == ST_PANEL) bd_copy16(o.r[0], lds + o.dst + 1024 * c, o.v[0], so + c * o.sub);
    else if constexpr (L == ST_ROWS) bd_copy16(o.r[0], lds + o.dst + 8192 * c, o.v[c], so);
    else bd_copy16(o.r[c], lds + o.dst + 8192 * c, o.v[c], so);
  }
}

// Lane offset, inside the operand's region, of the fragment of 16-row tile 0
// of a wave that starts at tile t0.
template <int L>
__device__ __forceinline__ int st_lane(int t0) {
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  if constexpr (L == ST_ROWS) return (16 * t0 + i) * ST_KB + 16 * (g ^ dt_swa(i));
  if constexpr (L == ST_PACK) return 1024 * t0 + 16 * lane;
  const int sig = (i >> 2) | ((g & 1) << 2);
  const int base = (8 * g + (i >> 2)) * BD_HPROW + 32 * sig + 8 * (i & 3);
  return (t0 >> 3) * BD_HP + (base ^ (32 * (t0 & 7)));
}

// Fragment of the wave's tile t (16 bytes).  ST_PANEL tiles of a wave lie in
// one half-panel and t0 is a multiple of the wave's tile count, so the tile
// index enters by XOR.
template <int L>
__device__ __forceinline__ u32x4 st_frag(const char* region, int lane_off, int t) {
  if constexpr (L == ST_PANEL) {
    const char* p = region + (lane_off ^ (32 * t));
    const s16x4 lo = dt_tr16(p), hi = dt_tr16(p + 4 * BD_HPROW);
    return __builtin_bit_cast(u32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    return *reinterpret_cast<const u32x4*>(region + lane_off + 1024 * t);
  }
}

__device__ __forceinline__ f32x4 st_mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  return mfma16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c);
}
__device__ __forceinline__ i32x4 st_mfma(const u32x4& a, const u32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c,
                                               0, 0, 0);
}

// Tile configuration.  NP phases of operands follow one another along K (the
// input gradient sums two products).  SPLIT: the 256 columns are 128 of one
// packed matrix and the same 128 of a second (gate and up products of one h
// column meet in one lane: acc[mt][t] and acc[mt][t + 4]).  KT: K is not a
// multiple of a stage; the fragments of a phase's last stage are zeroed past
// its end (ST_ROWS reads there what follows the row).
template <int MT_, int LA_, int LB_, typename AccT_, int NP_, bool SPLIT_, bool KT_>
struct StCfg {
  static constexpr int MT = MT_, LA = LA_, LB = LB_, NP = NP_;
  static constexpr bool SPLIT = SPLIT_, KT = KT_;
  typedef AccT_ Acc;
  static constexpr int BM = 64 * MT;
  typedef StOp<LA, BM> A;
  typedef StOp<LB, ST_BN> B;
  static constexpr int AB = A::BYTES, SLOT = AB + B::BYTES;   // columns follow the rows in a slot
  static constexpr int NS = MT == 4 ? 4 : 6;                   // ring slots (128 / 144 KB)
  static constexpr int LDS = NS * SLOT;
  static constexpr int CNT = A::C + B::C;                      // copies per wave per stage
  static_assert(MT == 2 || MT == 4, "128- or 256-row tiles");
  static_assert(NS % 2 == 0, "fragments alternate between two register sets");
};

template <class Cfg>
struct StCtx {
  typename Cfg::A a[Cfg::NP];
  typename Cfg::B b[Cfg::NP];
  int nst1;          // stages of a phase (all phases have the same K)
  int nst;           // stages in all
  int kvals;         // K of a phase in elements of 2 bytes (KT only)
  uint32_t lbase;
  int ao, bo;        // lane fragment offsets
};

template <class Cfg>
struct StFrag {
  u32x4 x[Cfg::MT], w[8];
};

template <class Cfg>
__device__ __forceinline__ void st_issue_all(const StCtx<Cfg>& c, int slot, int st) {
  uint32_t base = c.lbase;
  asm volatile("" : "+s"(base));   // one base, so that no address per slot stays in registers
  base += (uint32_t)(slot * Cfg::SLOT);
  if constexpr (Cfg::NP == 1) {
    st_issue(c.a[0], base, (uint32_t)st);
    st_issue(c.b[0], base + Cfg::AB, (uint32_t)st);
  } else {
    const bool second = st >= c.nst1;
    if (second) {
      st_issue(c.a[1], base, (uint32_t)(st - c.nst1));
      st_issue(c.b[1], base + Cfg::AB, (uint32_t)(st - c.nst1));
    } else {
      st_issue(c.a[0], base, (uint32_t)st);
      st_issue(c.b[0], base + Cfg::AB, (uint32_t)st);
    }
  }
}

// Whether this lane's k (8 bf16 from 8 g) lie past the end of stage st's phase.
template <class Cfg>
__device__ __forceinline__ bool st_past(const StCtx<Cfg>& c, int st) {
  if constexpr (!Cfg::KT) return false;
  const int s = Cfg::NP > 1 && st >= c.nst1 ? st - c.nst1 : st;
  return 32 * s + 8 * (int)((threadIdx.x & 63) >> 4) >= c.kvals;
}

template <class Cfg>
__device__ __forceinline__ void st_read_x(const StCtx<Cfg>& c, const char* slot, bool zero, StFrag<Cfg>& f) {
#pragma unroll
  for (int mt = 0; mt < Cfg::MT; ++mt) {
    f.x[mt] = st_frag<Cfg::LA>(slot, c.ao, mt);
    if (Cfg::KT && zero) f.x[mt] = u32x4{0u, 0u, 0u, 0u};
  }
}
template <class Cfg>
__device__ __forceinline__ void st_read_w(const StCtx<Cfg>& c, const char* slot, bool zero, int t,
                                          StFrag<Cfg>& f) {
  const int tt = Cfg::SPLIT ? (t & 3) + 8 * (t >> 2) : t;
  f.w[t] = st_frag<Cfg::LB>(slot + Cfg::AB, c.bo, tt);
  if (Cfg::KT && zero) f.w[t] = u32x4{0u, 0u, 0u, 0u};
}

template <int CNT>
__device__ __forceinline__ void st_sync_n(int n) {
  if (n >= 5) bd_sync<5 * CNT>();
  else bd_sync_n<CNT>(n);
}

// Step st (slot J): F holds its fragments.  Wait for stage st + 1 and meet the
// other waves (all have read slot J), refill slot J with stage st + NS, then
// read stage st + 1 into G while F is multiplied.
template <int J, bool GUARD, class Cfg>
__device__ __forceinline__ void st_step(const StCtx<Cfg>& c, char* ring, int st, StFrag<Cfg>& F, StFrag<Cfg>& G,
                                        typename Cfg::Acc (&acc)[Cfg::MT][8]) {
  constexpr int NS = Cfg::NS, MT = Cfg::MT;
  if (GUARD && st >= c.nst) return;
  const bool next = !GUARD || st + 1 < c.nst;
  if (next) {
    if (!GUARD) bd_sync<(NS - 2) * Cfg::CNT>();
    else st_sync_n<Cfg::CNT>(min(c.nst - 2 - st, NS - 2));
    if (!GUARD || st + NS < c.nst) st_issue_all(c, J % NS, st + NS);
  }
  __builtin_amdgcn_sched_barrier(0);
  const char* slot = ring + ((J + 1) % NS) * Cfg::SLOT;
  const bool zero = st_past(c, st + 1);
  if (next) st_read_x(c, slot, zero, G);
#pragma unroll
  for (int t = 0; t < 8; ++t) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt][t] = st_mfma(F.w[t], F.x[mt], acc[mt][t]);
    if (next) st_read_w(c, slot, zero, t, G);
  }
  if (next && !Cfg::KT) {
    __builtin_amdgcn_sched_group_barrier(0x100, Cfg::LA == ST_PANEL ? 2 * MT : MT, 0);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      __builtin_amdgcn_sched_group_barrier(0x008, MT, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, Cfg::LB == ST_PANEL ? 2 : 1, 0);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <int J, bool GUARD, class Cfg>
__device__ __forceinline__ void st_trip(const StCtx<Cfg>& c, char* ring, int st, StFrag<Cfg>& F, StFrag<Cfg>& G,
                                        typename Cfg::Acc (&acc)[Cfg::MT][8]) {
  st_step<J, GUARD>(c, ring, st + J, F, G, acc);
  if constexpr (J + 1 < Cfg::NS) st_trip<J + 1, GUARD>(c, ring, st, G, F, acc);
}

// The wave's fragment offsets and the ring's address (operands and stage
// counts are the caller's).
template <class Cfg>
__device__ __forceinline__ void st_setup(StCtx<Cfg>& c, char* ring) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  c.lbase = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(dt_lds_t*)ring);
  c.ao = st_lane<Cfg::LA>(Cfg::MT * (wave & 3));
  c.bo = st_lane<Cfg::LB>(Cfg::SPLIT ? 4 * (wave >> 2) : 8 * (wave >> 2));
}

template <class Cfg>
__device__ __forceinline__ void st_clear(typename Cfg::Acc (&acc)[Cfg::MT][8]) {
#pragma unroll
  for (int a = 0; a < Cfg::MT; ++a)
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[a][t] = typename Cfg::Acc{};
}

// acc += the product over c.nst stages.  No copy of this wave may be
// outstanding and every wave must be done with the ring.
template <class Cfg>
__device__ __forceinline__ void st_accum(const StCtx<Cfg>& c, char* ring, typename Cfg::Acc (&acc)[Cfg::MT][8]) {
  constexpr int NS = Cfg::NS;
  if (c.nst <= 0) return;
  for (int j = 0; j < NS; ++j)
    if (j < c.nst) st_issue_all(c, j, j);
  st_sync_n<Cfg::CNT>(min(c.nst - 1, NS - 1));
  StFrag<Cfg> F, G;
  const bool zero = st_past(c, 0);
  st_read_x(c, ring, zero, F);
#pragma unroll
  for (int t = 0; t < 8; ++t) st_read_w(c, ring, zero, t, F);
  int st = 0;
  for (; st + 2 * NS <= c.nst; st += NS) st_trip<0, false>(c, ring, st, F, G, acc);
  st_trip<0, true>(c, ring, st, F, G, acc);
  st_trip<0, true>(c, ring, st + NS, F, G, acc);
}

// ---------------------------------------------------------------------------
// row blocks of expert segments
// ---------------------------------------------------------------------------
constexpr int ST_MAXN = 1024;   // experts at most
constexpr int ST_GM = 8;        // row blocks of one expert that run together

struct StTile {
  int e, r0, R, nt;   // expert, first row, valid rows, column block
};

// pre[j] = row blocks of experts 0 .. j, bm rows each (segments of at most lo
// rows have none); returns their total.
// All threads call; the caller separates the next use of pre by a barrier.
__device__ __forceinline__ int st_prefix(const int32_t* __restrict__ offsets, int n, int bm, int* pre, int lo = 0) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int j0 = 0; j0 < n; j0 += 64) {
      const int j = j0 + lane;
      const int cnt = j < n ? offsets[j + 1] - offsets[j] : 0;
      int x = cnt > lo ? (cnt + bm - 1) / bm : 0;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(x, off);
        if (lane >= off) x += y;
      }
      if (j < n) pre[j] = carry + x;
      carry += __shfl(x, 63);
    }
    if (lane == 0) pre[ST_MAXN] = carry;
  }
  __syncthreads();
  return pre[ST_MAXN];
}

// Tile L of (row blocks) * ntn: an expert's tiles follow one another, in groups
// of ST_GM row blocks that run through the column blocks together, so that
// neighbouring tiles share weight columns and an expert's rows in an L2.
__device__ __forceinline__ StTile st_tile_at(int L, const int32_t* __restrict__ offsets, int n, int ntn, int bm,
                                             const int* pre) {
  int lo = 0, hi = n - 1;
  const int q = L / ntn;   // first e with pre[e] > q
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] > q) hi = mid; else lo = mid + 1;
  }
  const int first = lo ? pre[lo - 1] : 0;
  const int nrb = pre[lo] - first;
  const int local = L - first * ntn;
  const int mg = local / (ST_GM * ntn);
  const int rem = local - mg * ST_GM * ntn;
  const int gsz = min(ST_GM, nrb - mg * ST_GM);
  const int nt = rem / gsz;
  const int mb = mg * ST_GM + (rem - nt * gsz);
  const int o = offsets[lo];
  StTile t;
  t.e = __builtin_amdgcn_readfirstlane(lo);
  t.r0 = __builtin_amdgcn_readfirstlane(o + mb * bm);
  t.R = __builtin_amdgcn_readfirstlane(min(bm, offsets[lo + 1] - o - mb * bm));
  t.nt = __builtin_amdgcn_readfirstlane(nt);
  return t;
}

// The tiles [begin, end) of `total` that workgroup b of G takes, every `step`-th:
// each XCD (workgroup id mod 8 on this part) gets one contiguous range.
struct StRange {
  int begin, end, step;
};
__device__ __forceinline__ StRange st_range(int total, int b, int G) {
  if (G & 7) return StRange{b, total, G};
  const int x = b & 7, per = total >> 3, more = total & 7;
  const int first = x * per + min(x, more);
  return StRange{first + (b >> 3), first + per + (x < more ? 1 : 0), G >> 3};
}

}  // namespace moe
