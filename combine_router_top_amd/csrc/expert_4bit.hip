// Products of bf16 rows with 4-bit weights that have a scale, and perhaps a zero
// point, for each group of 32, 64 or 128 along K in each output channel, and the
// SwiGLU expert FFNs built from them.
//
//   W[k,j] = (q[k,j] - z[k/G,j]) s[k/G,j]         q, z in 0 .. 15 (z = 8 without zero points)
//   gemm   C = rnd(A W)
//   expert h = rnd(SiLU(x W1) (x W3)), y = rnd(h W2)
//
// Two forms of the product, by what either takes (w4_plan).  Streams, for few rows, read
// every weight once, straight into registers.  A group's part of a sum is
// s (sum x q - z sum x).  The matrix cores take q as the bf16 number (16 + q) / 4096, which is
// exact and costs one masked or of the packed bits (q is the upper mantissa of a number in
// 2^-8 .. 2^-7), so that with X = sum x / 4096 over the group
//
//   part = sum x (16 + q) / 4096,   C = 4096 sum s (part - (16 + z) X)
//
// X is one more product, with 1/4096.  All of it is fp32: no weight is ever rounded.  The
// offset makes the terms of a part about five times larger than those of the result, two
// bits of fp32's 24.  The 1/4096 keeps both of a group's sums, of up to 128 terms of 31 |x|,
// below the largest |x|, so that no part overflows; every bf16 x times (16 + q) / 4096 is a
// multiple of 2^-145, which fp32 holds, and what is summed last are multiples of 2^-149, so
// that results are off by up to 2^-137 for each group.  Tiles, for many rows: w4_tile.h.
//
// Packed weights: blocks of 16 columns x 128 K, 1 KB, one 16-byte load per lane and an
// operand of four MFMA k-steps after the masked ors: [N/16][K/128][64 lanes][4 words],
// lane 16 a + c holding column c, word s its k = 32 s + 8 a .. + 7, value 2 p + h at
// bits 16 h + 4 p, the word then rotated left by 3 bits to where the mantissas want it.
#include <stdint.h>

#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "w4.h"

namespace moe {

// ---------------------------------------------------------------------------
// quantiser and packing (once per set of weights)
// ---------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ float w4_load(const void* p, int64_t i) {
  return BF16 ? bf16_to_f32(reinterpret_cast<const bf16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

// Scales and zero points, one thread per group and column.  A group that holds an
// infinity or a NaN gets that as its scale, so that its products are no plausible numbers.
// (32 x 7168 x 2048 in bf16: 164 us, 5.7 TB/s.)
template <bool BF16>
__global__ __launch_bounds__(256) void w4_scales(const void* __restrict__ w, int K, int N, int G, int groups,
                                                 bf16_t* __restrict__ scale, uint8_t* __restrict__ zero) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)groups * N) return;
  const int grp = (int)(id / N), col = (int)(id - (int64_t)grp * N);
  const int64_t base = (int64_t)blockIdx.y * K * N + col;
  float lo = 0.f, hi = 0.f;
  uint32_t top = 0;
  for (int k = grp * G; k < min(K, grp * G + G); k += 8) {   // K is a multiple of 8
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = w4_load<BF16>(w, base + (int64_t)(k + u) * N);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      top = max(top, __float_as_uint(v[u]) & 0x7FFFFFFFu);
      lo = fminf(lo, v[u]);
      hi = fmaxf(hi, v[u]);
    }
  }
  const int64_t at = (int64_t)blockIdx.y * groups * N + id;
  const float big = __uint_as_float(top);
  // (a range past fp32's largest value by halves: elsewhere it is the one step documented)
  const float range = hi - lo;
  float s = !zero ? big / 7.0f : range < INFINITY ? range / 15.0f : (0.5f * hi - 0.5f * lo) / 7.5f;
  if (top >= 0x7F800000u) s = big;
  scale[at] = (bf16_t)cvt_bf16x2(s, 0.f);
  if (zero) {
    s = bf16_to_f32(scale[at]);
    zero[at] = s > 0.f && s < INFINITY ? (uint8_t)fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : (uint8_t)8;
  }
}

// One packed block per wave.  MODE 0: values 0 .. 15 as bytes [n][K][N] (higher bits are
// dropped); 1: bf16, 2: fp32 weights, quantised with the scales and zero points.
// (32 x 7168 x 2048 from bf16: 560 us, half of it the exact divisions; from bytes 290.)
template <int MODE>
__global__ __launch_bounds__(256) void w4_pack(const void* __restrict__ w, const bf16_t* __restrict__ scale,
                                               const uint8_t* __restrict__ zero, int K, int N, int G, int groups,
                                               int kb, int nt, u32x4* __restrict__ out) {
  const int lane = threadIdx.x & 63, c = lane & 15, a = lane >> 4;
  const int64_t blk = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (blk >= (int64_t)kb * nt) return;
  const int tn = (int)(blk / kb), tk = (int)(blk - (int64_t)tn * kb);
  const int col = 16 * tn + c;
  // all loads before the first use: of positions past the end, the last ones' in their place
  const int cl = min(col, N - 1);
  const int64_t base = (int64_t)blockIdx.y * K * N + cl, gbase = (int64_t)blockIdx.y * groups * N + cl;
  float x[4][8], sc[4], z[4];
  uint32_t b[4][8];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k0 = min(W4_KB * tk + 32 * s + 8 * a, K - 8);   // K is a multiple of 8, a group of 32
    const int64_t g = gbase + (int64_t)(k0 / G) * N;
    sc[s] = MODE ? bf16_to_f32(scale[g]) : 0.f;
    z[s] = MODE && zero ? (float)zero[g] : 8.f;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      if (MODE == 0) b[s][v] = reinterpret_cast<const uint8_t*>(w)[base + (int64_t)(k0 + v) * N];
      else x[s][v] = w4_load<MODE == 1>(w, base + (int64_t)(k0 + v) * N);
    }
  }
  u32x4 o;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    uint32_t word = 0;
    const bool live = MODE && sc[s] > 0.f && sc[s] < INFINITY;
    const float by = live ? sc[s] : 1.f;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      uint32_t q;
      if (MODE == 0) q = b[s][v] & 15u;
      else q = live ? (uint32_t)fminf(fmaxf(rintf(x[s][v] / by) + z[s], zero ? 0.f : 1.f), 15.f) : (uint32_t)z[s];
      word |= q << (16 * (v & 1) + 4 * (v >> 1));
    }
    if (col >= N || W4_KB * tk + 32 * s + 8 * a >= K) word = 0;
    o[s] = (word << 3) | (word >> 29);
  }
  out[((int64_t)blockIdx.y * kb * nt + blk) * 64 + lane] = o;
}

// ---------------------------------------------------------------------------
// streams
// ---------------------------------------------------------------------------
template <bool F32OUT>
__device__ __forceinline__ void w4_store(void* c, int64_t at, const float (&o)[4]) {
  if (F32OUT) *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(c) + at) = f32x4{o[0], o[1], o[2], o[3]};
  else
    *reinterpret_cast<u32x2*>(reinterpret_cast<bf16_t*>(c) + at) =
        u32x2{cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3])};
}

// The value of lane N of a row of 16 lanes in all of them; n is a constant after unrolling.
__device__ __forceinline__ uint32_t row_lane(uint32_t v, int n) {
  switch (n) {
#define ROW_LANE(N) \
  case N: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x150 + N, 0xf, 0xf, false);
    ROW_LANE(0) ROW_LANE(1) ROW_LANE(2) ROW_LANE(3) ROW_LANE(4) ROW_LANE(5) ROW_LANE(6) ROW_LANE(7)
    ROW_LANE(8) ROW_LANE(9) ROW_LANE(10) ROW_LANE(11) ROW_LANE(12) ROW_LANE(13) ROW_LANE(14)
#undef ROW_LANE
    default: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x15F, 0xf, 0xf, false);
  }
}

// Up to 16 MT rows o .. o + R - 1 against NT 16-column tiles (GATED: NT / 2 of each
// matrix).  The KS waves split K evenly by blocks; each loads its blocks straight into a
// ring of RB sets of registers, RB - 1 ahead of their use, and the fp32 sums meet in LDS in
// wave order.  GPB: groups of a block.  A lane needs the scales of four columns of each tile
// and group, the same for 16 lanes: each of the 16 loads another tile's or group's, and
// DPP hands them round (a load instruction occupies the address unit 16 cycles, whatever
// its lanes share).
template <int MT, int NT, bool GATED, bool F32OUT, int KS, int GPB, bool ZERO, int RB>
__device__ __forceinline__ void w4_stream_block(const W4Args& p, int e, int o, int R, f32x4* red, int stride) {
  constexpr int NH = GATED ? NT / 2 : NT, SPG = 4 / GPB;   // k-steps of a group
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile0 = (int)blockIdx.x * NH;
  const uint32_t run = (uint32_t)p.kb * 1024u;
  const int per = (p.kb + KS - 1) / KS, s0 = wave * per, ns = max(0, min(per, p.kb - s0));
  const int kend = min(p.K, (s0 + ns) * W4_KB);   // rows read zeros from there on
  const int64_t ge = (int64_t)e * p.groups * p.N;
  const uint32_t gsize = (uint32_t)p.groups * (uint32_t)p.N;
  constexpr int MATS = GATED ? 2 : 1;
  __amdgpu_buffer_rsrc_t rb[NT], rs[MATS], rz[MATS];
  uint32_t zsize[MATS];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const char* base = GATED && t >= NH ? p.b3 : p.b1;
    const int nt = min(tile0 + t % NH, p.ntiles - 1);
    rb[t] = gc_rsrc(base + ((int64_t)e * p.ntiles + nt) * run + (int64_t)s0 * 1024, (uint32_t)ns * 1024u);
  }
#pragma unroll
  for (int m = 0; m < MATS; ++m) {
    const uint8_t* z = m ? p.z3 : p.z1;
    rs[m] = gc_rsrc((m ? p.s3 : p.s1) + ge, gsize * 2u);
    zsize[m] = z ? gsize : 0u;
    rz[m] = gc_rsrc(z ? z + ge : (const uint8_t*)p.a, zsize[m]);
  }
  // lane i of a row loads tile i / GPB and group i % GPB
  static_assert(NH * GPB <= 16, "a lane for each tile and group");
  const int scol = 16 * (tile0 + min(i / GPB, NH - 1)) + 4 * g;
  const uint32_t vs = scol < p.N ? (uint32_t)(i % GPB) * (uint32_t)p.N + (uint32_t)scol : GC_OOR >> 1;
  const uint32_t asize = (uint32_t)R * (uint32_t)p.K * 2u;
  const __amdgpu_buffer_rsrc_t ra = gc_rsrc(p.a + (int64_t)o * p.K, asize);
  uint32_t va[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
    va[mt] = 16 * mt + i < R ? ((uint32_t)(16 * mt + i) * (uint32_t)p.K + 8u * (uint32_t)g) * 2u : GC_OOR;
  const uint32_t vb = 16u * (uint32_t)lane;
  // what is subtracted, X times: 16 and the zero point, 8 where there are none (they read as zeros)
  const float zb1 = p.z1 ? -16.f : -24.f, zb3 = GATED && p.z3 ? -16.f : -24.f;

  const uint32_t mask = w4_mask(), bits = w4_bits();
  f32x4 acc[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[mt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 w[RB][NT], x[RB][MT][4];
  u32x2 sc[RB][MATS];
  uint32_t zp[RB][MATS];
  auto load = [&](int h, int b) {   // block b of this wave; of one past its last, rows and weights are zeros
#pragma unroll
    for (int t = 0; t < NT; ++t)
      w[h][t] = __builtin_amdgcn_raw_buffer_load_b128(rb[t], vb, st_offset((uint32_t)b * 1024u, (uint32_t)ns * 1024u), 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = (s0 + b) * W4_KB + 32 * q;
      const bool in = k + 8 * g < kend;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        x[h][mt][q] = __builtin_amdgcn_raw_buffer_load_b128(ra, in ? va[mt] : GC_OOR, st_offset((uint32_t)k * 2u, asize), 0);
    }
    const uint32_t row = (uint32_t)((s0 + b) * GPB) * (uint32_t)p.N;
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      sc[h][m] = __builtin_amdgcn_raw_buffer_load_b64(rs[m], vs * 2u, st_offset(row * 2u, gsize * 2u), 0);
      if (ZERO) zp[h][m] = __builtin_amdgcn_raw_buffer_load_b32(rz[m], vs, st_offset(row, zsize[m]), 0);
    }
  };
  auto multiply = [&](int h) {
    const bf16x8 unit =   // 1/4096
        __builtin_bit_cast(bf16x8, u32x4{0x39803980u, 0x39803980u, 0x39803980u, 0x39803980u});
#pragma unroll
    for (int u = 0; u < GPB; ++u) {
      f32x4 X[MT], part[MT][NT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        X[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NT; ++t) part[mt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int q = u * SPG; q < (u + 1) * SPG; ++q) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) X[mt] = mfma16(unit, __builtin_bit_cast(bf16x8, x[h][mt][q]), X[mt]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const u32x4 f = w4_unpack(w[h][t][q], mask, bits);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) part[mt][t] = st_mfma(f, x[h][mt][q], part[mt][t]);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int m = GATED && t >= NH, from = t % NH * GPB + u;
        const u32x2 s2 = u32x2{row_lane(sc[h][m][0], from), row_lane(sc[h][m][1], from)};
        const uint32_t zq = ZERO ? row_lane(zp[h][m], from) : 0u;
        const float s[4] = {bf16_lo(s2[0]), bf16_hi(s2[0]), bf16_lo(s2[1]), bf16_hi(s2[1])};
        const float zb = GATED && t >= NH ? zb3 : zb1;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float z = ZERO ? zb - (float)((zq >> (8 * r)) & 255u) : -24.f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) acc[mt][t][r] = fmaf(s[r], fmaf(z, X[mt][r], part[mt][t][r]), acc[mt][t][r]);
        }
      }
    }
  };
  if (ns > 0) {
#pragma unroll
    for (int h = 0; h + 1 < RB; ++h) load(h, h);
    for (int b = 0; b < ns; b += RB) {
#pragma unroll
      for (int h = 0; h < RB; ++h) {
        load((h + RB - 1) % RB, b + h + RB - 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(h);   // a block past the last adds zeros
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[wave * stride + (mt * NT + t) * 64 + lane] = acc[mt][t];
  __syncthreads();
  for (int j = wave; j < MT * NH; j += KS) {
    const int mt = j / NH, t = j - mt * NH;
    const f32x4* at = red + (mt * NT + t) * 64 + lane;
    f32x4 p1 = at[0], p3 = at[GATED ? NH * 64 : 0];
#pragma unroll
    for (int v = 1; v < KS; ++v) {
      p1 += at[v * stride];
      if (GATED) p3 += at[v * stride + NH * 64];
    }
    const int row = 16 * mt + i, col = 16 * (tile0 + t) + 4 * g;
    if (row >= R || col >= p.N) continue;
    float v4[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) v4[r] = GATED ? silu_mul(4096.f * p1[r], 4096.f * p3[r]) : 4096.f * p1[r];
    w4_store<F32OUT>(p.c, (int64_t)(o + row) * p.N + col, v4);
  }
}

// All rows of a segment, 16 MT at a time, the blocks dealt out over gridDim.z
// workgroups; longer segments read their weights again for each block, from the caches.
// K is dealt out over KS waves, each with a run of whole packed blocks, which are operands
// as they are: a weight goes from memory to its product without LDS, and the waves' sums meet
// there at the end.  Bound by memory where there are many weights (32 experts of
// 7168 x 2048, 4 rows each: 82 us for the gated pair's 484 MB, 45 for the other's 242), by the
// latency of a few loads in turn where there are few (1 x 7168 x 2048: 6.2 us for 8 MB).
template <int MT, int NT, bool GATED, bool F32OUT, int KS, int GPB, bool ZERO, int RB>
__global__ __launch_bounds__(64 * KS) void w4_stream(W4Args p) {
  __shared__ __attribute__((aligned(16))) f32x4 red[KS][MT * NT][64];
  const int e = blockIdx.y;
  int o;
  const int R = w4_rows(p, e, o);
  constexpr int stride = MT * NT * 64;
  const int step = 16 * MT * (int)gridDim.z;
  for (int r0 = 16 * MT * (int)blockIdx.z; r0 < R; r0 += step) {
    if (r0 >= step) __syncthreads();   // the sums before have been read
    if (MT == 1 || R - r0 <= 16)
      w4_stream_block<1, NT, GATED, F32OUT, KS, GPB, ZERO, RB>(p, e, o + r0, min(16, R - r0), &red[0][0][0], stride);
    else w4_stream_block<MT, NT, GATED, F32OUT, KS, GPB, ZERO, RB>(p, e, o + r0, min(16 * MT, R - r0), &red[0][0][0], stride);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <bool GATED, bool F32OUT, int GPB, bool ZERO>
static hipError_t launch_4bit_stream(const W4Args& p, const W4Plan& plan, hipStream_t st) {
  auto go = [&](auto kernel, int cols, int ks) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((p.N + cols - 1) / cols), (unsigned)p.n, (unsigned)plan.blocks), dim3(64 * ks),
                       0, st, p);
    return hipGetLastError();
  };
  constexpr int NT = GATED ? 2 : 1, WIDE = GATED ? 32 : 64;
  if constexpr (!GATED)
    if (plan.ahead)
      return plan.low ? go(w4_stream<1, 4, GATED, F32OUT, 4, GPB, ZERO, 2>, WIDE, 4)
                      : go(w4_stream<2, 4, GATED, F32OUT, 4, GPB, ZERO, 2>, WIDE, 4);
  if (plan.wide)
    return plan.low ? go(w4_stream<1, 4, GATED, F32OUT, 8, GPB, ZERO, 1>, WIDE, 8)
                    : go(w4_stream<2, 4, GATED, F32OUT, 4, GPB, ZERO, 1>, WIDE, 4);
  if (plan.low)
    return plan.waves == 16 ? go(w4_stream<1, NT, GATED, F32OUT, 16, GPB, ZERO, 1>, 16, 16)
                            : go(w4_stream<1, NT, GATED, F32OUT, 8, GPB, ZERO, 1>, 16, 8);
  return go(w4_stream<2, NT, GATED, F32OUT, 8, GPB, ZERO, 1>, 16, 8);
}

// What a plan says, for the shape it was made for.
template <bool GATED, bool F32OUT>
static hipError_t launch_4bit(const W4Args& p, const W4Plan& plan, int group, int64_t rows_max, hipStream_t st) {
  if (plan.tiles)
    return GATED ? launch_4bit_tiles_up(p, group, plan.bm, rows_max, st)
                 : launch_4bit_tiles_down(p, group, plan.bm, rows_max, F32OUT, st);
  const bool zero = p.z1 || (GATED && p.z3);
  auto with = [&](auto gpb) {
    return zero ? launch_4bit_stream<GATED, F32OUT, gpb(), true>(p, plan, st)
                : launch_4bit_stream<GATED, F32OUT, gpb(), false>(p, plan, st);
  };
  return group == 32   ? with(std::integral_constant<int, 4>{})
         : group == 64 ? with(std::integral_constant<int, 2>{})
                       : with(std::integral_constant<int, 1>{});
}

// ---------------------------------------------------------------------------
// what the tiles take: rows in fp16, exponents of rows and columns
// ---------------------------------------------------------------------------
// Exponent k that puts |v| in 2^(top-1) .. 2^top; 0 for zero, an infinity or a NaN.
__device__ __forceinline__ int w4_exponent(uint32_t bits, int top) {
  if (bits == 0 || bits >= 0x7F800000u) return 0;
  return top - __builtin_amdgcn_frexp_expf(__uint_as_float(bits));
}

struct W4Columns {
  const bf16_t* s;   // [n][groups][N]
  int32_t* k;        // [n][N]
  int groups, N;
};
struct W4Prepare {
  const bf16_t* a;
  bf16_t* out;            // fp16 bits, K padded with zeros to whole blocks
  int32_t* kr;
  int64_t rows;
  const int32_t* limit;   // device row count, or NULL
  int K, n;
  W4Columns m[2];
};

constexpr int WP_U = 4;   // 8-value pieces a thread keeps between the two passes
constexpr int WP_COLS = 256;   // columns of a workgroup
typedef uint32_t u32x4_by8 __attribute__((ext_vector_type(4), aligned(8)));   // scales begin at 8 bytes

// Columns [c, c + WP_COLS) of an expert: thread (lane of 32, part of 8) takes 8 of them and
// every 8th group.
__device__ __forceinline__ void w4_columns(const W4Columns& m, int64_t e, int c, uint32_t (*part)[WP_COLS]) {
  const int lane = threadIdx.x & 31, by = threadIdx.x >> 5, col = c + 8 * lane;
  uint32_t top[8] = {};
  if (col < m.N) {
    const bf16_t* s = m.s + e * m.groups * m.N + col;
#pragma unroll 4
    for (int g = by; g < m.groups; g += 8) {
      const u32x4_by8 v = *reinterpret_cast<const u32x4_by8*>(s + (int64_t)g * m.N);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        top[2 * j] = max(top[2 * j], v[j] & 0x7FFFu);
        top[2 * j + 1] = max(top[2 * j + 1], (v[j] >> 16) & 0x7FFFu);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[by][8 * lane + j] = top[j];
  __syncthreads();
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) most = max(most, part[j][threadIdx.x]);
  if (c + (int)threadIdx.x < m.N) m.k[e * m.N + c + threadIdx.x] = w4_exponent(most << 16, 11);
}

// The first workgroups take the columns, the others rows (grid-stride).  Bound by memory:
// 4096 x 4096 rows and 14336 columns 15.6 us, 4.3 TB/s.
// A row with an infinity or a NaN holds a NaN afterwards, and so does every product of it.
__global__ __launch_bounds__(256) void w4_prepare(W4Prepare p, int col_blocks) {
  if ((int)blockIdx.x < col_blocks) {
    __shared__ uint32_t part[8][WP_COLS];
    int64_t at = blockIdx.x;
    int i = 0;
    for (; i < 2; ++i) {
      const int64_t here = (int64_t)p.n * ((p.m[i].N + WP_COLS - 1) / WP_COLS);
      if (at < here) break;
      at -= here;
    }
    const W4Columns m = p.m[i];
    const int per = (m.N + WP_COLS - 1) / WP_COLS;
    w4_columns(m, at / per, (int)(at % per) * WP_COLS, part);
    return;
  }
  const int first = (int)blockIdx.x - col_blocks, row_blocks = (int)gridDim.x - col_blocks;
  __shared__ uint32_t part[2][4];
  const int nv = p.K / 8;
  const int64_t rows = p.limit ? min(p.rows, (int64_t)*p.limit) : p.rows;
  int flip = 0;
  for (int64_t row = first; row < rows; row += row_blocks, flip ^= 1) {
    const u32x4* src = reinterpret_cast<const u32x4*>(p.a + row * p.K);
    u32x4 keep[WP_U];
    uint32_t top = 0;   // largest magnitude, as bf16 bits in either half
    auto see = [&](const u32x4& v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(v[j] & 0x7FFFu, (v[j] >> 16) & 0x7FFFu));
    };
#pragma unroll
    for (int u = 0; u < WP_U; ++u)
      if ((int)threadIdx.x + 256 * u < nv) keep[u] = src[threadIdx.x + 256 * u];
#pragma unroll
    for (int u = 0; u < WP_U; ++u)
      if ((int)threadIdx.x + 256 * u < nv) see(keep[u]);
    for (int v = threadIdx.x + 256 * WP_U; v < nv; v += 256) see(src[v]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
    if ((threadIdx.x & 63) == 0) part[flip][threadIdx.x >> 6] = top;
    __syncthreads();   // alternating halves: the next row's writes meet no reader of this one
    top = max(max(part[flip][0], part[flip][1]), max(part[flip][2], part[flip][3]));
    const int k = w4_exponent(top << 16, 15);
    const bool bad = top >= 0x7F80u;
    if (threadIdx.x == 0) p.kr[row] = k;
    const int nvp = (p.K + W4_KB - 1) / W4_KB * (W4_KB / 8);
    u32x4* dst = reinterpret_cast<u32x4*>(p.out + row * (8 * (int64_t)nvp));
    auto convert = [&](const u32x4& v) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a = __builtin_ldexpf(bf16_lo(v[j]), k), b = __builtin_ldexpf(bf16_hi(v[j]), k);
        if (bad) a = b = NAN;
        o[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
      }
      return o;
    };
#pragma unroll
    for (int u = 0; u < WP_U; ++u)
      if ((int)threadIdx.x + 256 * u < nv) dst[threadIdx.x + 256 * u] = convert(keep[u]);
    for (int v = threadIdx.x + 256 * WP_U; v < nv; v += 256) dst[v] = convert(src[v]);
    if ((int)threadIdx.x < nvp - nv) dst[nv + threadIdx.x] = u32x4{0, 0, 0, 0};
  }
}

static hipError_t launch_prepare(W4Prepare p, hipStream_t st) {
  int64_t cols = 0;
  for (const W4Columns& m : p.m) cols += (int64_t)p.n * ((m.N + WP_COLS - 1) / WP_COLS);
  const int rows = (int)std::min<int64_t>(p.rows, 8 * (int64_t)device_cus());
  hipLaunchKernelGGL(w4_prepare, dim3((unsigned)(rows + cols)), dim3(256), 0, st, p, (int)cols);
  return hipGetLastError();
}

size_t packed_4bit_bytes(int n, int K, int N) {
  return (size_t)n * ((K + W4_KB - 1) / W4_KB) * ((N + 15) / 16) * 1024;
}

hipError_t launch_pack_4bit(int n, int K, int N, const void* w, void* packed, hipStream_t st) {
  const int kb = (K + W4_KB - 1) / W4_KB, nt = (N + 15) / 16;
  hipLaunchKernelGGL(w4_pack<0>, dim3((unsigned)(((int64_t)kb * nt + 3) / 4), (unsigned)n), dim3(256), 0, st, w,
                     (const bf16_t*)nullptr, (const uint8_t*)nullptr, K, N, 32, 0, kb, nt, (u32x4*)packed);
  return hipGetLastError();
}

hipError_t launch_quantize_4bit(int n, int K, int N, int group, int dtype, const void* w, void* packed, void* scale,
                                void* zero, hipStream_t st) {
  const int kb = (K + W4_KB - 1) / W4_KB, nt = (N + 15) / 16, groups = (K + group - 1) / group;
  const dim3 g1((unsigned)(((int64_t)groups * N + 255) / 256), (unsigned)n);
  const dim3 g2((unsigned)(((int64_t)kb * nt + 3) / 4), (unsigned)n);
  auto scales = dtype == 1 ? w4_scales<true> : w4_scales<false>;
  auto pack = dtype == 1 ? w4_pack<1> : w4_pack<2>;
  hipLaunchKernelGGL(scales, g1, dim3(256), 0, st, w, K, N, group, groups, (bf16_t*)scale, (uint8_t*)zero);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(pack, g2, dim3(256), 0, st, w, (const bf16_t*)scale, (const uint8_t*)zero, K, N, group, groups, kb, nt,
                     (u32x4*)packed);
  return hipGetLastError();
}

// The products of the parts of K, summed in their order.  (Without parts 256 rows of
// 7168 x 2048 take 74 us, with them 19, of which 3 here.)
template <bool F32OUT>
__global__ __launch_bounds__(256) void w4_join(const f32x4* __restrict__ sums, void* __restrict__ c, int64_t vecs, int parts) {
  const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (v >= vecs) return;
  f32x4 a = sums[v];
#pragma unroll 4
  for (int s = 1; s < parts; ++s) a += sums[v + s * vecs];
  if constexpr (F32OUT) ((f32x4*)c)[v] = a;
  else ((u32x2*)c)[v] = u32x2{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3])};
}

static W4Args w4_args(int n, int K, int N, int group) {
  W4Args p{};
  p.n = n;
  p.K = K;
  p.N = N;
  p.kb = (K + W4_KB - 1) / W4_KB;
  p.ntiles = (N + 15) / 16;
  p.groups = (K + group - 1) / group;
  p.parts = 1;
  p.per = p.kb;
  return p;
}

static size_t pad256(size_t v) { return (v + 255) / 256 * 256; }
static size_t w4_row_bytes(int64_t rows, int K) { return (size_t)rows * ((K + W4_KB - 1) / W4_KB) * (2 * W4_KB); }

static W4Plan gemm_plan(int M, int N, int K) {
  return w4_plan(device_cus(), W4Shape{false, false, 1, N, (K + W4_KB - 1) / W4_KB, M, M, M});
}

size_t gemm_4bit_ws_bytes(int M, int N, int K) {
  const W4Plan plan = gemm_plan(M, N, K);
  const int parts = plan.parts;
  if (M == 0 || !plan.tiles) return 0;
  return pad256(w4_row_bytes(M, K)) + pad256((size_t)M * 4) + pad256((size_t)N * 4) + (parts > 1 ? (size_t)parts * M * N * 4 : 0);
}

hipError_t launch_gemm_4bit(int M, int N, int K, int group, const void* a, const void* packed, const void* scale,
                            const void* zero, void* c, int out_dtype, void* ws, hipStream_t st) {
  const W4Plan plan = gemm_plan(M, N, K);
  W4Args p = w4_args(1, K, N, group);
  p.M = M;
  p.a = (const bf16_t*)a;
  p.b1 = (const char*)packed;
  p.s1 = (const bf16_t*)scale;
  p.z1 = (const uint8_t*)zero;
  p.c = c;
  if (plan.tiles) {
    bf16_t* rows = (bf16_t*)ws;
    int32_t* kr = (int32_t*)((char*)ws + pad256(w4_row_bytes(M, K)));
    int32_t* kc = (int32_t*)((char*)kr + pad256((size_t)M * 4));
    const hipError_t e = launch_prepare(
        W4Prepare{p.a, rows, kr, M, nullptr, K, 1, {W4Columns{p.s1, kc, p.groups, N}, W4Columns{}}}, st);
    if (e != hipSuccess) return e;
    p.a = rows;
    p.kr = kr;
    p.k1 = kc;
    if (plan.parts > 1) {
      char* sums = (char*)kc + pad256((size_t)N * 4);
      p.parts = plan.parts;
      p.per = plan.per;
      p.part = (int64_t)M * N * 4;
      p.c = sums;
      const hipError_t t = launch_4bit_tiles_down(p, group, plan.bm, M, true, st);
      if (t != hipSuccess) return t;
      const int64_t vecs = (int64_t)M * N / 4;
      auto join = out_dtype == 1 ? w4_join<false> : w4_join<true>;
      hipLaunchKernelGGL(join, dim3((unsigned)((vecs + 255) / 256)), dim3(256), 0, st, (const f32x4*)sums, c, vecs, plan.parts);
      return hipGetLastError();
    }
  }
  return out_dtype == 1 ? launch_4bit<false, false>(p, plan, group, M, st) : launch_4bit<false, true>(p, plan, group, M, st);
}

struct W4Expert {
  W4Plan up, down;
  size_t x, h, krx, krh, k1, k3, k2, total;   // places in the workspace
};
static W4Expert expert_plan(const Prob& p) {
  W4Expert w;
  const int64_t mean = p.tk() / p.E, all = p.tk() * p.n / p.E;
  w.up = w4_plan(device_cus(), W4Shape{true, true, p.n, p.f, (p.d + W4_KB - 1) / W4_KB, mean, all, p.T});
  w.down = w4_plan(device_cus(), W4Shape{false, true, p.n, p.d, (p.f + W4_KB - 1) / W4_KB, mean, all, p.T});
  size_t o = 0;
  auto take = [&](bool wanted, size_t bytes) {
    const size_t at = o;
    o += wanted ? pad256(bytes) : 0;
    return at;
  };
  w.x = take(w.up.tiles, w4_row_bytes(p.rows_max, p.d));
  w.krx = take(w.up.tiles, (size_t)p.rows_max * 4);
  w.k1 = take(w.up.tiles, (size_t)p.n * p.f * 4);
  w.k3 = take(w.up.tiles, (size_t)p.n * p.f * 4);
  w.h = take(w.down.tiles, w4_row_bytes(p.rows_max, p.f));
  w.krh = take(w.down.tiles, (size_t)p.rows_max * 4);
  w.k2 = take(w.down.tiles, (size_t)p.n * p.d * 4);
  w.total = o;
  return w;
}
size_t expert_4bit_ws_bytes(const Prob& p) { return expert_plan(p).total; }

hipError_t launch_expert_4bit(const Prob& p, int group, const void* x, const int32_t* offsets, const Weights4& w1,
                              const Weights4& w3, const Weights4& w2, void* h, void* y, void* ws, hipStream_t st) {
  const W4Expert w = expert_plan(p);
  char* at = (char*)ws;
  const int32_t* rows = offsets + p.n;   // rows behind the last segment are not read
  hipError_t e;
  W4Args a = w4_args(p.n, p.d, p.f, group);
  a.offsets = offsets;
  a.a = (const bf16_t*)x;
  a.b1 = (const char*)w1.w;
  a.s1 = (const bf16_t*)w1.scale;
  a.z1 = (const uint8_t*)w1.zero;
  a.b3 = (const char*)w3.w;
  a.s3 = (const bf16_t*)w3.scale;
  a.z3 = (const uint8_t*)w3.zero;
  a.c = h;
  W4Args b = w4_args(p.n, p.f, p.d, group);
  b.offsets = offsets;
  b.a = (const bf16_t*)h;
  b.b1 = (const char*)w2.w;
  b.s1 = (const bf16_t*)w2.scale;
  b.z1 = (const uint8_t*)w2.zero;
  b.c = y;
  if (w.up.tiles) {
    a.kr = (const int32_t*)(at + w.krx);
    a.k1 = (const int32_t*)(at + w.k1);
    a.k3 = (const int32_t*)(at + w.k3);
    W4Prepare q{a.a, (bf16_t*)(at + w.x), (int32_t*)(at + w.krx), p.rows_max, rows, p.d, p.n,
                {W4Columns{a.s1, (int32_t*)(at + w.k1), a.groups, p.f}, W4Columns{a.s3, (int32_t*)(at + w.k3), a.groups, p.f}}};
    if ((e = launch_prepare(q, st)) != hipSuccess) return e;
    a.a = q.out;
  }
  if ((e = launch_4bit<true, false>(a, w.up, group, p.rows_max, st)) != hipSuccess) return e;
  if (w.down.tiles) {
    b.kr = (const int32_t*)(at + w.krh);
    b.k1 = (const int32_t*)(at + w.k2);
    W4Prepare q{b.a, (bf16_t*)(at + w.h), (int32_t*)(at + w.krh), p.rows_max, rows, p.f, p.n,
                {W4Columns{b.s1, (int32_t*)(at + w.k2), b.groups, p.d}, W4Columns{}}};
    if ((e = launch_prepare(q, st)) != hipSuccess) return e;
    b.a = q.out;
  }
  return launch_4bit<false, false>(b, w.down, group, p.rows_max, st);
}

}  // namespace moe
