// Tiles of the 4-bit products (gfx950): up to 192 rows x 256 columns (gated: 128 of each
// matrix), four waves, one on each SIMD, each with all rows of 64 columns.
//
// What bounds them is how much else than matrix products a wave issues, and the power the
// products draw: a 16 x 16 x 32 product takes 9 to 10 ns of a SIMD under load, one vector
// instruction beside it is nearly free, each further one of the same wave costs 1 to 2 ns
// (products alone 380 us of 4096 x 4096 x 14336, the whole tile kernel 410 to 490 us, by how
// long it has run, where 563 us were taken by eight waves of 96 x 64, which make every weight
// twice).  So:
//   - the tiles work in fp16, where a weight is made complete before it is multiplied, and no
//     sum is scaled later.  Rows come with a power of two that puts their largest value in
//     2^14 .. 2^15: every bf16 value within 2^-31 of it is exact in fp16, smaller ones are off by
//     less than 2^-38 of it.  Scales likewise, by columns, with their largest in 2^10 .. 2^11:
//     exact within 2^-27 of it, else off by less than 2^-34 of it.  The epilogue takes both
//     powers out again.
//   - without zero points, q becomes the fp16 number 16 + q by one masked or (two values),
//     and one packed fma with s and -24 s gives (q - 8) s: exactly, since 8-bit scales times
//     -8 .. 7 and times 24 fit fp16's 11 bits.  With zero points, 128 + q, an exact
//     subtraction and a product, which rounds odd multiples above 8 to 11 bits (by up to
//     2^-11 relative, once per weight; a bf16 output is rounded by up to 2^-8).
//   - an operand of 8 weights costs 12 (15) instructions and serves all row tiles, and these
//     instructions, the copies and the reads are dealt out between the products.
//
// Heights are 64, 96, 128, 160 or 192 rows, for each tile by its actual rows.  K runs in steps of
// 64: rows in a ring of three slots, packed blocks of 128 K with their scales in a ring of two,
// all copied from memory straight into LDS.  While a k-step of 32 is multiplied, the operands of
// the next are made, and a row fragment's registers take its successor as soon as they are
// free.  One barrier per step, once the first products of its second half are under way: by
// then every wave holds that half.  The next tile's first copies are issued before this
// one's stores.
#pragma once

#include "w4.h"

namespace moe {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int GPB_, bool ZERO_, bool GATED_, bool F32OUT_>
struct W4Cfg {
  static constexpr int GPB = GPB_;
  static constexpr bool ZERO = ZERO_, GATED = GATED_, F32OUT = F32OUT_;
  static constexpr int WAVES = 4;
  static constexpr int NT = 4, NH = GATED ? 2 : 4;      // a wave's weight and output tiles
  static constexpr int COLS = GATED ? 128 : 256;        // output columns of a tile
  static constexpr int XSLOT = 192 * 128;               // 64 K of 192 rows
  static constexpr int WOFF = 3 * XSLOT;                // the packed blocks' ring
  // a slot of it: 16 blocks, a group's scales (512 bytes), its zero points (256, gated: 256 of
  // each matrix, half of them used)
  static constexpr int SOFF = 16 * 1024, ZROW = GATED ? 512 : 256, ZOFF = SOFF + GPB * 512;
  static constexpr int WSLOT = ZOFF + (ZERO ? GPB * ZROW : 0);
  static constexpr int LDS = WOFF + 2 * WSLOT;
  // copies of a wave: packed blocks, and pieces of 256 bytes of scales and zero points dealt
  // out over the waves (some twice, so that every wave issues as many)
  static constexpr int SP = 2 * GPB, PIECES = SP + (ZERO ? (GATED ? 2 : 1) * GPB : 0);
  static constexpr int WB = 16 / WAVES, CS = (PIECES + WAVES - 1) / WAVES, W = WB + CS;
  static_assert(LDS <= 160 * 1024, "LDS");
};

// 16 (4) bytes per lane from descriptor r at voff + soff to LDS at `lds` + at + 16 (4) lane.
template <int BYTES>
__device__ __forceinline__ void w4_copy(__amdgpu_buffer_rsrc_t r, uint32_t lds, int at, uint32_t voff, uint32_t soff) {
  if constexpr (BYTES == 16)
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds"
                 :: "s"(lds), "i"(at), "v"(voff), "s"(r), "s"(soff) : "memory", "m0", "scc");
  else
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dword %2, %3, %4 offen lds"
                 :: "s"(lds), "i"(at), "v"(voff), "s"(r), "s"(soff) : "memory", "m0", "scc");
}

// A 256-byte piece of a block's scales or zero points: group u, matrix or half of the columns hm.
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

// A tile: rows and columns, and the blocks of 128 K that are multiplied.
struct W4Tile : StTile {
  int b0, nb, part;   // first block, their number, which part of K that is
};

// What a wave copies of the weights of a tile.
template <class C>
struct W4Ctx {
  const char* w[2];        // packed runs of the tile's first columns (gated: of each matrix)
  uint32_t wsize;          // bytes from there to the end of the expert's
  uint32_t woff[C::WB];    // lane offsets of its runs
  const char* s[C::CS];    // its pieces of scales or zero points of the first block
  uint32_t ssize[C::CS];   // bytes from there to the end of the matrix's, 0 for zero points that it has not
  uint32_t sstep[C::CS];   // bytes between blocks
  uint32_t sdst[C::CS];    // where in a slot
};

__device__ __forceinline__ const char* w4_scalar(const char* p) {   // descriptors are made of it
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const char*>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at) |
                                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) << 32);
}

template <class C>
__device__ __forceinline__ void w4_setup(const W4Args& p, const W4Tile& t, W4Ctx<C>& c) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t run = (uint32_t)p.kb * 1024u;
  const int first = C::COLS / 16 * t.nt, most = p.ntiles - 1 - first;
  const int64_t eo = ((int64_t)t.e * p.ntiles + first) * run + 1024 * t.b0;
  c.w[0] = w4_scalar(p.b1 + eo);
  c.w[1] = w4_scalar((C::GATED ? p.b3 : p.b1) + eo);
  c.wsize = __builtin_amdgcn_readfirstlane((uint32_t)min((int64_t)(most + 1) * run, (int64_t)UINT32_MAX) - 1024u * (uint32_t)t.b0);
#pragma unroll
  for (int v = 0; v < C::WB; ++v) {   // packed tiles wave, wave + 4, .. (gated: the second half of the second matrix)
    const int at = wave + C::WAVES * v;
    c.woff[v] = (uint32_t)min(C::GATED ? at % 8 : at, most) * run + 16u * (threadIdx.x & 63);
  }
  const int64_t go = (int64_t)t.e * p.groups * p.N + C::COLS * t.nt;
#pragma unroll
  for (int v = 0; v < C::CS; ++v) {
    const W4Piece q = w4_piece<C>(wave + C::WAVES * v);
    const bool m = C::GATED && q.hm;
    const uint8_t* zp = m ? p.z3 : p.z1;
    const uint32_t row = (uint32_t)p.N * (q.zero ? 1u : 2u);   // bytes of a group
    const uint32_t skip = row * (uint32_t)(q.u + t.b0 * C::GPB) + (C::GATED || q.zero ? 0u : 256u * (uint32_t)q.hm);
    const uint32_t size = q.zero && !zp ? 0u : (uint32_t)p.groups * row - (uint32_t)(C::COLS * t.nt) * (q.zero ? 1u : 2u);
    c.s[v] = w4_scalar((q.zero ? (const char*)(zp + go) : (const char*)((m ? p.s3 : p.s1) + go)) + skip);
    c.ssize[v] = __builtin_amdgcn_readfirstlane(size > skip ? size - skip : 0u);
    c.sstep[v] = __builtin_amdgcn_readfirstlane(row * (uint32_t)C::GPB);
    c.sdst[v] = __builtin_amdgcn_readfirstlane(q.dst);
  }
}

// Copy v (of W) of block b, one of the tile's, into the slot at LDS address `slot` (of this
// wave: slot + 1024 wave).  Groups that a last block has not, and zero points that the matrix
// has not, read zeros.
template <class C>
__device__ __forceinline__ void w4_issue(const W4Ctx<C>& c, uint32_t slot, int b, int v) {
  if (v < C::WB) {
    const __amdgpu_buffer_rsrc_t r = gc_rsrc(c.w[C::GATED && v >= C::WB / 2 ? 1 : 0], c.wsize);
    w4_copy<16>(r, slot + 1024 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), 1024 * C::WAVES * v, c.woff[v], (uint32_t)b * 1024u);
  } else {
    const int u = v - C::WB;
    w4_copy<4>(gc_rsrc(c.s[u], c.ssize[u]), slot + c.sdst[u], 0, 4u * (threadIdx.x & 63),
               st_offset((uint32_t)b * c.sstep[u], c.ssize[u]));
  }
}

__device__ __forceinline__ uint32_t w4_vreg(uint32_t v) {   // a constant that is no literal (w4_unpack)
  asm("" : "+v"(v));
  return v;
}
__device__ __forceinline__ uint32_t w4_sreg(uint32_t v) {
  asm("" : "+s"(v));
  return v;
}

// The rows' copies (fp16, of K padded to whole blocks), 8 rows of 64 K each: copy c of wave w
// takes rows 32 c + 8 w .. + 7.  Rows past the last one lie outside the descriptor and read
// zeros.
template <int X>
struct W4Rows {
  const char* base;
  uint32_t voff[X], size;
  __device__ __forceinline__ void of(const W4Args& p, const W4Tile& t, int rows) {
    const uint32_t ld = (uint32_t)p.kb * (2 * W4_KB);   // bytes of a row
    const int r = 8 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + ((threadIdx.x & 63) >> 3);
    base = w4_scalar((const char*)(p.a + (int64_t)t.r0 * (p.kb * W4_KB) + t.b0 * W4_KB));
#pragma unroll
    for (int c = 0; c < X; ++c) voff[c] = (uint32_t)(r + 32 * c) * ld + 16u * (uint32_t)((threadIdx.x & 7) ^ ((r >> 1) & 7));
    size = __builtin_amdgcn_readfirstlane((uint32_t)rows * ld - 2u * W4_KB * (uint32_t)t.b0);
  }
  __device__ __forceinline__ void issue(uint32_t slot, int st, int c) const {   // slot: of this wave
    w4_copy<16>(gc_rsrc(base, size), slot + 1024 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), 4096 * c, voff[c],
                (uint32_t)st * ST_KB);
  }
};

// As __builtin_amdgcn_mfma_f32_16x16x32_f16, with the sum held in place: of so many sums the
// compiler moves some at every turn of the loop.  What it would see to is seen to here: a
// vector instruction that writes an operand has two others between it and its product, and a
// sum is read only after w4_mfma_done().
__device__ __forceinline__ void w4_mfma(const u32x4& a, const u32x4& b, f32x4& c) {
  asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void w4_mfma_done() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// Row tiles of a tile of `rows` rows.
__device__ __forceinline__ int w4_height(int rows) { return rows <= 64 ? 4 : min(2 * ((rows + 31) / 32), 12); }

// The first copies of a tile: two blocks of the weights, three steps of the rows.  Copies run
// ahead of the products, past the last block or step too: they take the last one again, which
// is not multiplied (bounding every offset by its buffer instead took 0.7% more).
template <class C>
__device__ __forceinline__ void w4_begin(const W4Args& p, const W4Tile& t, const W4Ctx<C>& c, uint32_t lbase) {
  const uint32_t ld = (uint32_t)p.kb * (2 * W4_KB);
  const int X = w4_height(t.R) / 2;
  W4Rows<1> x;
  x.of(p, t, t.R);
  const __amdgpu_buffer_rsrc_t r = gc_rsrc(x.base, x.size);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int u = 0; u < C::W; ++u) w4_issue(c, lbase + C::WOFF + b * C::WSLOT, st_upto(b, t.nb), u);
  for (int u = 0; u < X; ++u)
#pragma unroll
    for (int j = 0; j < 3; ++j)
      w4_copy<16>(r, lbase + 1024 * wave + 4096 * u, j * C::XSLOT, x.voff[0] + (uint32_t)(32 * u) * ld,
                  (uint32_t)st_upto(j, 2 * t.nb) * ST_KB);
}

// A tile's product for L row tiles a wave.
template <class C, int L>
struct W4Wave {
  static constexpr int NT = C::NT, NH = C::NH;
  f32x4 acc[L][NT];
  u32x4 x[L];              // rows of a k-step
  u32x4 w[NT];             // packed words of a block
  u32x4 f[2][NT];          // operands of a k-step and of the next
  uint32_t S[NT], Z[NT];   // scale and addend of the group that operands are made of, twice each
  int k[NT];               // exponents of this lane's columns
  uint32_t mask, bits, zmul, zbase[2];
  int xo, at0;             // lane offsets in a slot: rows, and the wave's first column tile

  static __device__ __forceinline__ int matrix(int t) { return C::GATED ? t / NH : 0; }
  __device__ __forceinline__ int tile(int t) const { return at0 + (C::GATED ? t % NH + 8 * (t / NH) : t); }   // of the slot's 16

  __device__ __forceinline__ void read_x(const char* slot, int ks, int m) {
    x[m] = st_frag<ST_ROWS>(slot, xo, ks, m);
  }
  __device__ __forceinline__ void read_w(const char* slot) {
#pragma unroll
    for (int t = 0; t < NT; ++t) w[t] = *reinterpret_cast<const u32x4*>(slot + 1024 * tile(t) + 16 * (threadIdx.x & 63));
  }
  // Scales and zero points of the block's group u, as they are, and the operands' made of them.
  __device__ __forceinline__ void read_scales(const char* slot, int u) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int col = 16 * tile(t) + (int)(threadIdx.x & 15);   // of the slot's 256
      S[t] = *reinterpret_cast<const uint16_t*>(slot + C::SOFF + 512 * u + 2 * col);
      if constexpr (C::ZERO)
        Z[t] = *reinterpret_cast<const uint8_t*>(slot + C::ZOFF + C::ZROW * u + col + (C::GATED ? 128 * matrix(t) : 0));
    }
  }
  __device__ __forceinline__ void make_scale(int t) {
    const float s = __builtin_ldexpf(__uint_as_float(S[t] << 16), k[t]);
    S[t] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(s, s));   // exact: 8 bits
    if constexpr (C::ZERO) Z[t] = Z[t] * zmul + zbase[matrix(t)];            // -(128 + z), twice
    else Z[t] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, S[t]) * f16x2{(_Float16)-24, (_Float16)-24});
  }
  // Numbers p and p + 4 of the packed word of k-step n, as operand values of buffer b, in steps.
  __device__ __forceinline__ void pick(int b, int t, int n, int p) {
    const uint32_t word = w[t][n];
    const int r = (C::ZERO ? 4 * p : 4 * p + 29) & 31;
    f[b][t][p] = ((r ? __builtin_amdgcn_alignbit(word, word, r) : word) & mask) | bits;
  }
  __device__ __forceinline__ void less(int b, int t, int p) {
    f[b][t][p] = __builtin_bit_cast(uint32_t, half2(f[b][t][p]) + half2(Z[t]));
  }
  __device__ __forceinline__ void weigh(int b, int t, int p) {
    const f16x2 v = half2(f[b][t][p]), s = half2(S[t]);
    f[b][t][p] = __builtin_bit_cast(uint32_t, C::ZERO ? v * s : __builtin_elementwise_fma(v, s, half2(Z[t])));
  }
  static __device__ __forceinline__ f16x2 half2(uint32_t v) { return __builtin_bit_cast(f16x2, v); }
  // Step h of PARTS for two pairs of numbers, two instructions each (a sum is not
  // followed at once by the product that takes it, which would wait).
  static constexpr int PARTS = C::ZERO ? 4 : 3;
  __device__ __forceinline__ void part(int b, int n, int h) {
    const int t = h / (2 * PARTS), p = h / PARTS % 2 * 2;
    switch (h % PARTS) {
      case 0: pick(b, t, n, p); break;
      case 1: pick(b, t, n, p + 1); break;
      case PARTS - 1: weigh(b, t, p); weigh(b, t, p + 1); break;
      default: less(b, t, p); less(b, t, p + 1);
    }
  }
  // k-step Q of a block: products with f[Q & 1]; meanwhile the operands of the next from
  // the words w (SCALES: scales that were just read), and the rows of the next from (next, ks),
  // after `sync`, which comes once the first products are under way.  A product leaves room
  // for one or two vector instructions of its wave, more in a row hold up the next: so they
  // are dealt out, in a fixed order, and so are the COPIES copies, copy(0), copy(1), ..
  template <int Q, bool SCALES, int COPIES, class Sync, class Copy>
  __device__ __forceinline__ void kstep(const char* next, int ks, const Sync& sync, const Copy& copy) {
    constexpr int b = Q & 1, n = (Q + 1) & 3;
    constexpr int S0 = L > 4, MS = S0 + 1 + (L > 8), M0 = MS + 1, M1 = L - (L > 4);
    constexpr int H = 2 * PARTS * NT, A = M0 * NT, B = M1 * NT;   // halves, and the products beside which they are made
#pragma unroll
    for (int m = 0; m < L; ++m) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        w4_mfma(f[b][t], x[m], acc[m][t]);
        __builtin_amdgcn_sched_barrier(0);
        if (SCALES && m == MS) make_scale(t);
#pragma unroll
        for (int h = 0; h < H; ++h)
          if (A + h * (B - A) / H == m * NT + t) part(b ^ 1, n, h);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (m == S0) {
        sync();
#pragma unroll
        for (int j = 0; j <= S0; ++j) read_x(next, ks, j);
      }
      if (m > S0) {
        read_x(next, ks, m);   // into the registers just used
#pragma unroll
        for (int c = 0; c < COPIES; ++c)
          if (S0 + 1 + c * (L - 1 - S0) / (COPIES ? COPIES : 1) == m) copy(c);
      }
    }
  }
};

// Product of a tile whose first copies are under way; `after` begins the next one, once the
// ring is free, before this one's stores.
template <class C, int L, class After>
__device__ __forceinline__ void w4_tile_product(const W4Args& p, const W4Tile t, char* ring, const W4Ctx<C>& c,
                                                const After& after) {
  constexpr int NT = C::NT, NH = C::NH, GPB = C::GPB, X = L / 2;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lbase = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(dt_lds_t*)ring);
  W4Rows<X> xr;
  xr.of(p, t, min(t.R, 16 * L));
  W4Wave<C, L> v;
  v.xo = st_lane<ST_ROWS>(0);
  v.at0 = NH * wave;
  v.mask = w4_vreg(C::ZERO ? 0x00780078u : 0x03C003C0u);
  v.bits = w4_sreg(C::ZERO ? 0x58005800u : 0x4C004C00u);
  v.zmul = w4_sreg(0x00080008u);
  v.zbase[0] = w4_vreg(p.z1 ? 0xD800D800u : 0xD840D840u);   // without zero points: 8
  v.zbase[1] = w4_vreg(p.z3 ? 0xD800D800u : 0xD840D840u);
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int col = C::COLS * t.nt + 16 * (v.at0 + (C::GATED ? q % NH : q)) + i;
    v.k[q] = col < p.N ? (C::GATED && q >= NH ? p.k3 : p.k1)[(int64_t)t.e * p.N + col] : 0;
  }
#pragma unroll
  for (int m = 0; m < L; ++m)
#pragma unroll
    for (int q = 0; q < NT; ++q) v.acc[m][q] = f32x4{0.f, 0.f, 0.f, 0.f};
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): or the compiler waits for these loads in the loop
  st_sync<0>();
  const char* ws = ring + C::WOFF;   // slot of this block
#pragma unroll
  for (int m = 0; m < L; ++m) v.read_x(ring, 0, m);
  v.read_w(ws);
  v.read_scales(ws, 0);
#pragma unroll
  for (int q = 0; q < NT; ++q) v.make_scale(q);
#pragma unroll
  for (int h = 0; h < 2 * NT * v.PARTS; ++h) v.part(0, 0, h);
  uint32_t x0 = 0, x1 = C::XSLOT, x2 = 2 * C::XSLOT;   // slots of this step, the next and the one after
  uint32_t wo = 0;                                     // offset of this block's slot
  for (int b = 0; b < t.nb; ++b) {
    ws = ring + C::WOFF + wo;
    auto nothing = [](auto...) {};
    if (GPB == 4) v.read_scales(ws, 1);
    v.template kstep<0, GPB == 4, 0>(ring + x0, 1, nothing, nothing);
    if (GPB >= 2) v.read_scales(ws, GPB == 2 ? 1 : 2);
    // the next step's rows have arrived, this step's are in registers: their slot is refilled
    v.template kstep<1, GPB >= 2, X>(ring + x1, 0, [] { st_sync<C::W + X>(); },
                                     [&](int u) { xr.issue(lbase + x0, st_upto(2 * b + 3, 2 * t.nb), u); });
    if (GPB == 4) v.read_scales(ws, 3);
    v.template kstep<2, GPB == 4, 0>(ring + x1, 1, nothing, nothing);
    v.template kstep<3, true, C::W + X>(ring + x2, 0, [&] {
      st_sync<X>();
      v.read_w(ring + C::WOFF + C::WSLOT - wo);
      v.read_scales(ring + C::WOFF + C::WSLOT - wo, 0);
    }, [&](int u) {
      if (u < C::W) w4_issue(c, lbase + C::WOFF + wo, st_upto(b + 2, t.nb), u);
      else xr.issue(lbase + x1, st_upto(2 * b + 4, 2 * t.nb), u - C::W);
    });
    wo = C::WSLOT - wo;
    const uint32_t keep = x0;
    x0 = x2;
    x2 = x1;
    x1 = keep;
  }
  w4_mfma_done();
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");   // every wave is done with the ring

  const int col0 = C::COLS * t.nt + 16 * NH * wave;
  int kc[NT][4];   // exponents of the columns that this lane stores
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int col = min(col0 + 16 * (C::GATED ? q % NH : q) + 4 * g, p.N - 4);
    const i32x4 e = *reinterpret_cast<const i32x4*>((C::GATED && q >= NH ? p.k3 : p.k1) + (int64_t)t.e * p.N + col);
#pragma unroll
    for (int r = 0; r < 4; ++r) kc[q][r] = e[r];
  }
  int kr[L];
#pragma unroll
  for (int m = 0; m < L; ++m) kr[m] = p.kr[t.r0 + min(16 * m + i, t.R - 1)];
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): not after the copies that follow
  after();

  constexpr int ES = C::F32OUT ? 4 : 2;
  const StOut out = st_out((char*)p.c + t.part * p.part + (int64_t)t.r0 * p.N * ES, (int64_t)p.N * ES, t.R);
#pragma unroll
  for (int m = 0; m < L; ++m) {
    const int row = 16 * m + i;
    f32x4 o[NH];
#pragma unroll
    for (int q = 0; q < NH; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float a = __builtin_ldexpf(v.acc[m][q][r], -(kr[m] + kc[q][r]));
        if constexpr (C::GATED) o[q][r] = silu_mul(a, __builtin_ldexpf(v.acc[m][q + NT - NH][r], -(kr[m] + kc[q + NT - NH][r])));
        else o[q][r] = a;
      }
    if constexpr (C::F32OUT) {
#pragma unroll
      for (int q = 0; q < NH; ++q) {
        const int at = col0 + 16 * q + 4 * g;
        st_put(out, row, 4u * (uint32_t)at, at < p.N, __builtin_bit_cast(u32x4, o[q]));
      }
    } else {
#pragma unroll
      for (int q = 0; q < NH; q += 2) {
        const int at = col0 + 16 * q + 8 * g;
        st_put(out, row, 2u * (uint32_t)at, at < p.N, st_pack8(o[q], o[q + 1]));
      }
    }
  }
}

template <class C>
__global__ __launch_bounds__(64 * C::WAVES, 1) void w4_tile(W4Args p, int ntn, int bm) {
  __shared__ __attribute__((aligned(16))) char ring[C::LDS];
  const int blocks = p.offsets ? st_row_blocks(p.offsets, p.n, bm) : (p.M + bm - 1) / bm;
  const uint32_t lbase = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(dt_lds_t*)ring);
  const int tiles = blocks * ntn, total = tiles * p.parts;
  auto tile = [&](int L) {
    W4Tile t;
    t.part = p.parts > 1 ? st_div(L, tiles) : 0;
    L -= t.part * tiles;
    static_cast<StTile&>(t) = p.offsets ? st_tile_at(L, p.offsets, p.n, ntn, bm) : st_tile_of(L, 0, p.M, blocks, ntn, bm);
    t.b0 = t.part * p.per;
    t.nb = min(p.per, p.kb - t.b0);
    return t;
  };
  int L = st_first_tile();
  if (L >= total) return;
  W4Ctx<C> c;
  W4Tile t = tile(L);
  w4_setup<C>(p, t, c);
  w4_begin(p, t, c, lbase);
  for (;;) {
    const W4Tile now = t;
    L += (int)gridDim.x;
    auto after = [&] {
      if (L >= total) return;
      t = tile(L);
      w4_setup<C>(p, t, c);
      w4_begin(p, t, c, lbase);
    };
    switch (w4_height(now.R)) {
      case 4: w4_tile_product<C, 4>(p, now, ring, c, after); break;
      case 6: w4_tile_product<C, 6>(p, now, ring, c, after); break;
      case 8: w4_tile_product<C, 8>(p, now, ring, c, after); break;
      case 10: w4_tile_product<C, 10>(p, now, ring, c, after); break;
      default: w4_tile_product<C, 12>(p, now, ring, c, after);
    }
    if (L >= total) return;
  }
}

template <bool GATED, bool F32OUT, int GPB, bool ZERO>
static hipError_t launch_w4_tile(const W4Args& p, int bm, int64_t rows_max, hipStream_t st) {
  using C = W4Cfg<GPB, ZERO, GATED, F32OUT>;
  const int ntn = (p.N + C::COLS - 1) / C::COLS;
  hipLaunchKernelGGL(w4_tile<C>, st_row_grid(rows_max, p.n, bm / 64, ntn * p.parts), dim3(64 * C::WAVES), 0, st, p, ntn, bm);
  return hipGetLastError();
}

template <bool GATED, bool F32OUT>
static hipError_t launch_w4_tiles(const W4Args& p, int group, int bm, int64_t rows_max, hipStream_t st) {
  const bool zero = p.z1 || (GATED && p.z3);
  auto with = [&](auto gpb) {
    return zero ? launch_w4_tile<GATED, F32OUT, gpb(), true>(p, bm, rows_max, st)
                : launch_w4_tile<GATED, F32OUT, gpb(), false>(p, bm, rows_max, st);
  };
  return group == 32   ? with(std::integral_constant<int, 4>{})
         : group == 64 ? with(std::integral_constant<int, 2>{})
                       : with(std::integral_constant<int, 1>{});
}

}  // namespace moe
