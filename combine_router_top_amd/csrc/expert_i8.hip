// 8-bit integer products with a scale for each row and each output channel,
// and the SwiGLU expert FFNs built from them.
//
//   quantize_rows     s[m] = max_k |x[m,k]| / 127,  q[m,k] = rint(x[m,k] (127 (1 / max)))
//   quantize_weights  the same for each output channel of an expert's [K][N] weights
//   gemm_i8           C[m,n] = rnd((sum_k A[m,k] B[k,n]) sa[m] sb[n])
//   expert_gemm_i8    h = rnd(SiLU(x W1) (x W3)), y = rnd(h W2) with x and h
//                     quantised by rows and the weights by output channels
//
// The sums are exact: products of 8-bit values in int32, K < 131072.  A sum is
// therefore the same in any order, and the split of K over waves costs no
// reproducibility.  The only roundings are the quantisers', the conversion of a
// sum to fp32, two fp32 products and the store.
//
// Weights are packed once in the order the matrix cores take them: 1 KB blocks
// of 16 columns x 64 K, [N/16][K/64][4 k-groups][16 columns][16 k], zero past K
// and N.  A block is one 16-byte load per lane, contiguous over the wave, and
// is already an MFMA operand, so that a row-streaming kernel needs neither LDS
// nor a transpose, and the copies and reads of an LDS-staged tile are linear.
#include <stdint.h>

#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "seg_tile.h"

namespace moe {

// ---------------------------------------------------------------------------
// quantisers
// ---------------------------------------------------------------------------
// Factor of a row or channel with maximum `top`: 127 (1 / top), each operation
// rounded to fp32.  Below 2^-119 the factor would leave the fp32 range: such a
// row counts as zeros.  A row with an infinity or a NaN has the factor 0 and that
// value as its scale: every product with it is then NaN instead of a plausible
// number.
constexpr float Q_TINY = 0x1p-119f;
__device__ __forceinline__ float quant_factor(float top) { return top >= Q_TINY ? 127.0f * (1.0f / top) : 0.f; }
__device__ __forceinline__ float quant_scale(float top) { return top < Q_TINY ? 0.f : top / 127.0f; }

// max |v| by the bits, which order magnitudes as integers with NaN above infinity
// (a float maximum would drop a NaN).
__device__ __forceinline__ uint32_t top_of(uint32_t top, float v) { return max(top, __float_as_uint(v) & 0x7FFFFFFFu); }

// Four values q = rint(v inv) in the bytes of a word (|v inv| <= 127 up to one
// rounding, so the result fits int8; the conversion takes NaN, 0 times an infinity,
// to 0).
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float inv) {
  const uint32_t q0 = (uint32_t)(int)rintf(a * inv) & 255u, q1 = (uint32_t)(int)rintf(b * inv) & 255u;
  const uint32_t q2 = (uint32_t)(int)rintf(c * inv) & 255u, q3 = (uint32_t)(int)rintf(d * inv) & 255u;
  return q0 | (q1 << 8) | (q2 << 16) | (q3 << 24);
}

struct F8 {
  float v[8];
};
template <bool BF16>
__device__ __forceinline__ F8 load8(const void* p, int64_t i8) {
  F8 o;
  if (BF16) {
    const u32x4 w = reinterpret_cast<const u32x4*>(p)[i8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      o.v[2 * q] = bf16_lo(w[q]);
      o.v[2 * q + 1] = bf16_hi(w[q]);
    }
  } else {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[2 * i8], b = reinterpret_cast<const f32x4*>(p)[2 * i8 + 1];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      o.v[q] = a[q];
      o.v[4 + q] = b[q];
    }
  }
  return o;
}

constexpr int QR_U = 4;   // 8-value pieces a thread keeps between the two passes

// One workgroup per row (grid-stride): maximum, then the quantised row from
// the registers that the first pass filled (rows of up to 256 * 8 * QR_U
// values; the rest of a longer row is read again).  limit (or NULL): only rows
// below *limit.  Bound by its bytes: 4096 x 4096 bf16 in 10.6 us, 4.7 TB/s.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* __restrict__ x, int64_t rows, int K,
                                                            int64_t ldq, int8_t* __restrict__ q,
                                                            float* __restrict__ s, const int32_t* __restrict__ limit) {
  __shared__ uint32_t part[2][4];
  const int nv = K / 8;
  if (limit) rows = min(rows, (int64_t)*limit);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, flip ^= 1) {
    const char* src = reinterpret_cast<const char*>(x) + row * K * (BF16 ? 2 : 4);
    F8 keep[QR_U];
    uint32_t bits = 0;
#pragma unroll
    for (int u = 0; u < QR_U; ++u) {
      const int v = threadIdx.x + 256 * u;
      if (v < nv) keep[u] = load8<BF16>(src, v);
    }
#pragma unroll
    for (int u = 0; u < QR_U; ++u)
      if ((int)threadIdx.x + 256 * u < nv)
#pragma unroll
        for (int j = 0; j < 8; ++j) bits = top_of(bits, keep[u].v[j]);
    for (int v = threadIdx.x + 256 * QR_U; v < nv; v += 256) {
      const F8 o = load8<BF16>(src, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) bits = top_of(bits, o.v[j]);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) bits = max(bits, (uint32_t)__shfl_xor((int)bits, off));
    if ((threadIdx.x & 63) == 0) part[flip][threadIdx.x >> 6] = bits;
    __syncthreads();   // alternating halves: the next row's writes meet no reader of this one
    const float top = __uint_as_float(max(max(part[flip][0], part[flip][1]), max(part[flip][2], part[flip][3])));
    const float inv = quant_factor(top);
    if (threadIdx.x == 0) s[row] = quant_scale(top);
    u32x2* dst = reinterpret_cast<u32x2*>(q + row * ldq);
#pragma unroll
    for (int u = 0; u < QR_U; ++u) {
      const int v = threadIdx.x + 256 * u;
      const float* o = keep[u].v;
      if (v < nv) dst[v] = u32x2{quant4(o[0], o[1], o[2], o[3], inv), quant4(o[4], o[5], o[6], o[7], inv)};
    }
    for (int v = threadIdx.x + 256 * QR_U; v < nv; v += 256) {
      const F8 o = load8<BF16>(src, v);
      dst[v] = u32x2{quant4(o.v[0], o.v[1], o.v[2], o.v[3], inv), quant4(o.v[4], o.v[5], o.v[6], o.v[7], inv)};
    }
  }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return BF16 ? bf16_to_f32(reinterpret_cast<const bf16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

// Channel maxima of [n][K][N] weights: 64 columns per workgroup, K over 4
// groups of threads.  Done once per set of weights: 32 matrices of 7168 x 2048 in bf16
// take 1.41 ms with the packing (287 us of bytes at the copy rate), bound by 2-byte
// loads and, for a single matrix, by few workgroups (4096 x 14336: 339 us).
template <bool BF16>
__global__ __launch_bounds__(256) void channel_max_kernel(const void* __restrict__ w, int K, int N,
                                                            float* __restrict__ s) {
  __shared__ uint32_t part[4][64];
  const int col = blockIdx.x * 64 + (threadIdx.x & 63), grp = threadIdx.x >> 6;
  const int64_t base = (int64_t)blockIdx.y * K * N;
  uint32_t top = 0;
  if (col < N)
    for (int k = grp; k < K; k += 4) top = top_of(top, load1<BF16>(w, base + (int64_t)k * N + col));
  part[grp][threadIdx.x & 63] = top;
  __syncthreads();
  if (grp == 0 && col < N) {
    top = max(max(part[0][threadIdx.x], part[1][threadIdx.x]), max(part[2][threadIdx.x], part[3][threadIdx.x]));
    s[(int64_t)blockIdx.y * N + col] = __uint_as_float(top);
  }
}

// One packed block (16 columns x 64 K) per wave; MODE 0: int8 [n][K][N] as it
// is, 1: bf16, 2: fp32, both quantised with the channel's maximum in smax.  MODE 0 on
// 32 matrices of 7168 x 2048: 458 us, 2.05 TB/s, bound by its single-byte loads.
template <int MODE>
__global__ __launch_bounds__(256) void pack_kernel(const void* __restrict__ w, const float* __restrict__ smax, int K,
                                                   int N, int kt, int nt, u32x4* __restrict__ out) {
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int64_t blk = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (blk >= (int64_t)kt * nt) return;
  const int tn = (int)(blk / kt), tk = (int)(blk - (int64_t)tn * kt);
  const int col = 16 * tn + i, k0 = 64 * tk + 16 * g;
  const int64_t base = (int64_t)blockIdx.y * K * N;
  float inv = 0.f;
  if (MODE != 0 && col < N) {
    inv = quant_factor(smax[(int64_t)blockIdx.y * N + col]);
  }
  u32x4 o = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int b = 0; b < 16; ++b) {
    int v = 0;
    if (col < N && k0 + b < K) {
      const int64_t at = base + (int64_t)(k0 + b) * N + col;
      if (MODE == 0) v = reinterpret_cast<const int8_t*>(w)[at];
      else v = (int)rintf(load1<MODE == 1>(w, at) * inv);
    }
    o[b >> 2] |= ((uint32_t)v & 255u) << (8 * (b & 3));
  }
  out[((int64_t)blockIdx.y * kt * nt + blk) * 64 + lane] = o;
}

// Scales from channel maxima, in place.
__global__ __launch_bounds__(256) void scale_from_max_kernel(float* __restrict__ s, int64_t count) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < count) s[i] = quant_scale(s[i]);
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// What a product reads and writes.  Segments: rows [offsets[e], offsets[e+1])
// of expert e, or, without offsets, one segment of rows [0, M).
struct I8Args {
  const int8_t* a;        // [*][lda] bytes, row-major
  const float* sa;        // scale of each row
  const char* b1;         // packed weights [n][ntiles][kt] blocks
  const char* b3;         // second matrix of a gated product
  const float* s1;        // [n][N] channel scales
  const float* s3;
  void* c;                // [*][N]
  const int32_t* offsets;
  int n, M;               // experts; rows without offsets
  int lda, K, N;          // bytes per row of a, those that may be read (a multiple of 16), output columns
  int kt, ntiles;         // 64-K blocks and 16-column tiles of the packed weights
  int lo, hi;             // this launch takes segments with lo < rows <= hi (tiles: no upper bound)
};

__device__ __forceinline__ int i8_rows(const I8Args& p, int e, int& o) {
  int cnt;
  if (p.offsets) {
    o = p.offsets[e];
    cnt = p.offsets[e + 1] - o;
  } else {
    o = 0;
    cnt = p.M;
  }
  o = __builtin_amdgcn_readfirstlane(o);
  cnt = __builtin_amdgcn_readfirstlane(cnt);
  return cnt > p.lo && cnt <= p.hi ? cnt : 0;
}

// Four neighbouring columns of one output row.  Rounded by the hardware's conversion,
// as in the tiles: it keeps a NaN of any payload a NaN (a scale may hold any).
template <bool F32OUT>
__device__ __forceinline__ void i8_store(void* c, int64_t at, const float (&o)[4]) {
  if (F32OUT) *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(c) + at) = f32x4{o[0], o[1], o[2], o[3]};
  else
    *reinterpret_cast<u32x2*>(reinterpret_cast<bf16_t*>(c) + at) =
        u32x2{cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3])};
}

template <bool GATED>
__device__ __forceinline__ void i8_values(const i32x4& p1, const i32x4& p3, float sr, const f32x4& c1,
                                          const f32x4& c3, float (&o)[4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float a = (float)p1[r] * sr * c1[r];
    // the library's exponential and a true division, not silu_mul: h is
    // quantised next, where an ulp at a bf16 border can move a value by a whole
    // 8-bit step of its row
    o[r] = GATED ? a / (1.0f + expf(-a)) * ((float)p3[r] * sr * c3[r]) : a;
  }
}

// Tiles of 64 MT rows x 256 weight columns, or 64 x 128 (GATED: half as many
// output columns, of both matrices), for segments of more than `lo` rows.
// 4096 x 4096 x 14336: 218 us, 2.2 POPS; 32 experts of about 128 rows, gated
// 7168 x 2048: 206 us, the weights at 4.6 TB/s.
template <int MT, bool GATED, bool F32OUT>
using I8Cfg = StCfg<MT, ST_ROWS, ST_PACK, i32x4, 1, GATED,
                    MT * (MT == 1 ? 1 : 2) * (F32OUT ? 4 : 2) / (GATED ? 2 : 1)>;

template <int MT, bool GATED, bool F32OUT>
__global__ __launch_bounds__(ST_NT, 1) void i8_tile(I8Args p, int ntn) {
  using Cfg = I8Cfg<MT, GATED, F32OUT>;
  __shared__ __attribute__((aligned(16))) char ring[Cfg::LDS];
  // without offsets: one segment of M rows, ntn column blocks
  const int total = (p.offsets ? st_row_blocks(p.offsets, p.n, Cfg::BM, p.lo) : (p.M + Cfg::BM - 1) / Cfg::BM) * ntn;
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 3, wn = wave >> 2;
  const uint32_t run = (uint32_t)p.kt * 1024u;
  st_run<Cfg>(
      total, ring,
      [&](int L, StCtx<Cfg>& c) {
        const StTile t = p.offsets ? st_tile_at(L, p.offsets, p.n, ntn, Cfg::BM, p.lo)
                                   : st_tile_of(L, 0, p.M, (p.M + Cfg::BM - 1) / Cfg::BM, ntn, Cfg::BM);
        st_rows(c.a[0], p.a + (int64_t)t.r0 * p.lda, (uint32_t)p.lda, t.R, (uint32_t)p.K);
        const int64_t eo = (int64_t)t.e * p.ntiles * run;
        st_pack<GATED>(c.b[0], p.b1 + eo, GATED ? p.b3 + eo : nullptr, (GATED ? Cfg::BN / 32 : Cfg::BN / 16) * t.nt,
                       p.ntiles, run);
        c.nst = c.nst1 = (p.kt + 1) / 2;   // an odd last block meets zeros past its run
        return t;
      },
      [&](const StTile& t, typename Cfg::Acc& acc) {
        constexpr int ES = F32OUT ? 4 : 2;
        const StOut out = st_out((char*)p.c + (int64_t)t.r0 * p.N * ES, (int64_t)p.N * ES, t.R);
        float sr[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) sr[mt] = p.sa[t.r0 + min(16 * MT * wm + 16 * mt + i, t.R - 1)];
        const float* s1 = p.s1 + (int64_t)t.e * p.N;
        const float* s3 = GATED ? p.s3 + (int64_t)t.e * p.N : nullptr;
        const int col0 = (GATED ? Cfg::BN / 2 * t.nt + Cfg::WN / 2 * wn : Cfg::BN * t.nt + Cfg::WN * wn);
        constexpr int OT = GATED ? Cfg::NT / 2 : Cfg::NT;   // column tiles of output
#pragma unroll
        for (int k = 0; k < OT; k += 2) {
          f32x4 c1[2], c3[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = min(col0 + 16 * (k + h) + 4 * q, p.N - 4);
            c1[h] = *reinterpret_cast<const f32x4*>(s1 + col);
            c3[h] = GATED ? *reinterpret_cast<const f32x4*>(s3 + col) : c1[h];
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int row = 16 * MT * wm + 16 * mt + i;
            float x[4], y[4];
            i8_values<GATED>(acc[mt][k], acc[mt][GATED ? k + OT : k], sr[mt], c1[0], c3[0], x);
            i8_values<GATED>(acc[mt][k + 1], acc[mt][GATED ? k + OT + 1 : k + 1], sr[mt], c1[1], c3[1], y);
            if (F32OUT) {
              const int at = col0 + 16 * k + 4 * q;
              st_put(out, row, 4u * (uint32_t)at, at < p.N, __builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]}));
              st_put(out, row, 4u * (uint32_t)(at + 16), at + 16 < p.N,
                     __builtin_bit_cast(u32x4, f32x4{y[0], y[1], y[2], y[3]}));
            } else {
              const int at = col0 + 16 * k + 8 * q;
              st_put(out, row, 2u * (uint32_t)at, at < p.N, st_pack8(x, y));
            }
          }
        }
      });
}

// Short segments: a stream of the packed weights.  Workgroup (task, e) owns NT
// 16-column tiles (GATED: NT / 2 of each matrix); its KS waves split K evenly,
// each loads its blocks straight into MFMA operands, U stages ahead of their
// use, and the int32 sums meet in LDS.  Rows of A come through the caches.  Past
// its part of K a wave's weight descriptors read zeros, so that the loop needs
// no tail.  128 rows over 32 experts, 7168 x 2048: gated 155 us, the weights at 6.1
// TB/s, as fast as a plain streaming read.  One call multiplies up to 16 MT rows, o .. o + R - 1.
template <int MT, int NT, bool GATED, bool F32OUT, int KS, int U>
__device__ __forceinline__ void i8_stream_block(const I8Args& p, int e, int o, int R, i32x4* red, int stride) {
  constexpr int NH = GATED ? NT / 2 : NT;   // output column tiles
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile0 = (int)blockIdx.x * NH;
  const uint32_t run = (uint32_t)p.kt * 1024u;
  const int per = (p.kt + KS - 1) / KS, s0 = wave * per, ns = max(0, min(per, p.kt - s0));
  __amdgpu_buffer_rsrc_t rb[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const char* base = GATED && t >= NH ? p.b3 : p.b1;
    const int nt = min(tile0 + (GATED ? t % NH : t), p.ntiles - 1);
    rb[t] = gc_rsrc(base + ((int64_t)e * p.ntiles + nt) * run + (int64_t)s0 * 1024, (uint32_t)ns * 1024u);
  }
  // rows of A: the descriptor ends with the segment's last valid byte
  const __amdgpu_buffer_rsrc_t ra =
      gc_rsrc(p.a + (int64_t)o * p.lda, (uint32_t)(R - 1) * (uint32_t)p.lda + (uint32_t)p.K);
  uint32_t va[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
    va[mt] = (uint32_t)min(16 * mt + i, R - 1) * (uint32_t)p.lda + 16u * (uint32_t)g + 64u * (uint32_t)s0;
  const uint32_t vb = 16u * (uint32_t)lane;
  i32x4 acc[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[mt][t] = i32x4{0, 0, 0, 0};
  u32x4 w[2][U][NT], x[2][U][MT];
  auto load = [&](int h, int st) {
#pragma unroll
    for (int v = 0; v < U; ++v) {
#pragma unroll
      for (int t = 0; t < NT; ++t) w[h][v][t] = __builtin_amdgcn_raw_buffer_load_b128(rb[t], vb, (st + v) * 1024, 0);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) x[h][v][mt] = __builtin_amdgcn_raw_buffer_load_b128(ra, va[mt], (st + v) * 64, 0);
    }
  };
  auto multiply = [&](int h) {
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[mt][t] = st_mfma(w[h][v][t], x[h][v][mt], acc[mt][t]);
  };
  if (ns > 0) {
    load(0, 0);
    for (int st = 0; st < ns; st += 2 * U) {
      load(1, st + U);
      __builtin_amdgcn_sched_barrier(0);
      multiply(0);
      __builtin_amdgcn_sched_barrier(0);
      load(0, st + 2 * U);
      __builtin_amdgcn_sched_barrier(0);
      multiply(1);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[wave * stride + (mt * NT + t) * 64 + lane] = acc[mt][t];
  __syncthreads();
  const float* s1 = p.s1 + (int64_t)e * p.N;
  const float* s3 = GATED ? p.s3 + (int64_t)e * p.N : nullptr;
  for (int j = wave; j < MT * NH; j += KS) {
    const int mt = j / NH, t = j - mt * NH;
    const i32x4* at = red + (mt * NT + t) * 64 + lane;
    i32x4 p1 = at[0], p3 = at[GATED ? NH * 64 : 0];
#pragma unroll
    for (int v = 1; v < KS; ++v) {
      p1 += at[v * stride];
      if (GATED) p3 += at[v * stride + NH * 64];
    }
    const int row = 16 * mt + i, col = 16 * (tile0 + t) + 4 * g;
    if (row >= R || col >= p.N) continue;
    const f32x4 c1 = *reinterpret_cast<const f32x4*>(s1 + col);
    const f32x4 c3 = GATED ? *reinterpret_cast<const f32x4*>(s3 + col) : c1;
    float v4[4];
    i8_values<GATED>(p1, p3, p.sa[o + row], c1, c3, v4);
    i8_store<F32OUT>(p.c, (int64_t)(o + row) * p.N + col, v4);
  }
}

// All rows of a segment, 16 MT at a time, the blocks dealt out over gridDim.z
// workgroups (with MT = 2 a last block of up to 16 rows multiplies half as much); longer segments read their weights again for
// each block, from the caches.  MT = 1, for batches of up to 16 rows, holds fewer
// registers, hence more waves and loads in flight (8 rows, 4096 x 14336: 17
// against 23 us with the quantiser).
template <int MT, int NT, bool GATED, bool F32OUT, int KS, int U1, int U2>
__global__ __launch_bounds__(64 * KS) void i8_stream(I8Args p) {
  __shared__ __attribute__((aligned(16))) i32x4 red[KS][MT * NT][64];
  const int e = blockIdx.y;
  int o;
  const int R = i8_rows(p, e, o);
  constexpr int stride = MT * NT * 64;
  const int step = 16 * MT * (int)gridDim.z;
  for (int r0 = 16 * MT * (int)blockIdx.z; r0 < R; r0 += step) {
    if (r0 >= step) __syncthreads();   // the sums before have been read
    if (MT == 1 || R - r0 <= 16)
      i8_stream_block<1, NT, GATED, F32OUT, KS, U1>(p, e, o + r0, min(16, R - r0), &red[0][0][0], stride);
    else i8_stream_block<2, NT, GATED, F32OUT, KS, U2>(p, e, o + r0, min(32, R - r0), &red[0][0][0], stride);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// What i8_plan says for a product of these rows.
template <bool GATED, bool F32OUT>
static hipError_t launch_product(I8Args p, int64_t mean, int64_t all, int64_t most, int64_t rows_max, hipStream_t st) {
  const I8Plan plan = i8_plan(device_cus(), I8Shape{GATED, p.offsets != nullptr, p.n, p.N, p.kt, mean, all, most});
  if (plan.stream) {
    p.lo = 0;
    p.hi = plan.tiles ? I8_THIN : INT32_MAX;
    auto go = [&](auto kernel, int cols, int ks) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)((p.N + cols - 1) / cols), (unsigned)p.n, (unsigned)plan.blocks),
                         dim3(64 * ks), 0, st, p);
      return hipGetLastError();
    };
    constexpr int NT = GATED ? 2 : 1;
    hipError_t e;
    if (plan.low)
      e = plan.wide ? go(i8_stream<1, 4, GATED, F32OUT, 4, 4, 4>, GATED ? 32 : 64, 4)
                    : go(i8_stream<1, NT, GATED, F32OUT, 8, 4, 4>, 16, 8);
    else
      e = plan.wide ? go(i8_stream<2, 4, GATED, F32OUT, 4, 4, 3>, GATED ? 32 : 64, 4)
                    : go(i8_stream<2, NT, GATED, F32OUT, 8, 4, 4>, 16, 8);
    if (e != hipSuccess || !plan.tiles) return e;
  }
  p.lo = plan.stream ? I8_THIN : 0;
  return st_with_height(plan.height, [&](auto height) {
    constexpr int H = height(), cols = i8_cols(GATED, H);
    const int ntn = (p.N + cols - 1) / cols;
    hipLaunchKernelGGL((i8_tile<H, GATED, F32OUT>), st_row_grid(rows_max, p.n, H, ntn), dim3(ST_NT), 0, st, p, ntn);
    return hipGetLastError();
  });
}

hipError_t launch_quantize_rows(const void* x, int dtype, int64_t rows, int K, int64_t ldq, void* q, float* s,
                                const int32_t* limit, hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>(rows, 8 * (int64_t)device_cus()));
  if (dtype == 1)
    hipLaunchKernelGGL(quantize_rows_kernel<true>, grid, dim3(256), 0, st, x, rows, K, ldq, (int8_t*)q, s, limit);
  else
    hipLaunchKernelGGL(quantize_rows_kernel<false>, grid, dim3(256), 0, st, x, rows, K, ldq, (int8_t*)q, s, limit);
  return hipGetLastError();
}

size_t packed_i8_bytes(int n, int K, int N) {
  return (size_t)n * ((K + 63) / 64) * ((N + 15) / 16) * 1024;
}

hipError_t launch_pack_i8(int n, int K, int N, const void* w, void* packed, hipStream_t st) {
  const int kt = (K + 63) / 64, nt = (N + 15) / 16;
  hipLaunchKernelGGL(pack_kernel<0>, dim3((unsigned)(((int64_t)kt * nt + 3) / 4), (unsigned)n), dim3(256), 0, st, w,
                     (const float*)nullptr, K, N, kt, nt, (u32x4*)packed);
  return hipGetLastError();
}

hipError_t launch_quantize_weights(int n, int K, int N, int dtype, const void* w, void* packed, float* s,
                                   hipStream_t st) {
  const int kt = (K + 63) / 64, nt = (N + 15) / 16;
  const dim3 g1((unsigned)((N + 63) / 64), (unsigned)n), g2((unsigned)(((int64_t)kt * nt + 3) / 4), (unsigned)n);
  if (dtype == 1) {
    hipLaunchKernelGGL(channel_max_kernel<true>, g1, dim3(256), 0, st, w, K, N, s);
    hipLaunchKernelGGL(pack_kernel<1>, g2, dim3(256), 0, st, w, (const float*)s, K, N, kt, nt, (u32x4*)packed);
  } else {
    hipLaunchKernelGGL(channel_max_kernel<false>, g1, dim3(256), 0, st, w, K, N, s);
    hipLaunchKernelGGL(pack_kernel<2>, g2, dim3(256), 0, st, w, (const float*)s, K, N, kt, nt, (u32x4*)packed);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t count = (int64_t)n * N;
  hipLaunchKernelGGL(scale_from_max_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, st, s, count);
  return hipGetLastError();
}

hipError_t launch_gemm_i8(int M, int N, int K, const void* a, const float* sa, const void* packed, const float* sb,
                          void* c, int out_dtype, hipStream_t st) {
  I8Args p{};
  p.a = (const int8_t*)a;
  p.sa = sa;
  p.b1 = (const char*)packed;
  p.s1 = sb;
  p.c = c;
  p.n = 1;
  p.M = M;
  p.lda = K;
  p.K = K;
  p.N = N;
  p.kt = (K + 63) / 64;
  p.ntiles = (N + 15) / 16;
  return out_dtype == 1 ? launch_product<false, false>(p, M, M, M, M, st) : launch_product<false, true>(p, M, M, M, M, st);
}

static size_t pad256(size_t v) { return (v + 255) / 256 * 256; }
static int pad64(int v) { return (v + 63) / 64 * 64; }

size_t expert_i8_ws_bytes(const Prob& p) {
  // quantised rows of x and of h (64-byte rows), and their scales
  return pad256((size_t)p.rows_max * pad64(p.d)) + pad256((size_t)p.rows_max * pad64(p.f)) +
         2 * pad256((size_t)p.rows_max * 4);
}

hipError_t launch_expert_i8(const Prob& p, const void* x, const int32_t* offsets, const void* q1, const float* s1,
                            const void* q3, const float* s3, const void* q2, const float* s2, void* h, void* y,
                            void* ws, hipStream_t st) {
  char* at = (char*)ws;
  int8_t* xq = (int8_t*)at;
  int8_t* hq = (int8_t*)(at += pad256((size_t)p.rows_max * pad64(p.d)));
  float* sx = (float*)(at += pad256((size_t)p.rows_max * pad64(p.f)));
  float* sh = (float*)(at += pad256((size_t)p.rows_max * 4));
  const int32_t* rows = offsets + p.n;   // rows behind the last segment are not read
  const int64_t mean = p.tk() / p.E, all = p.tk() * p.n / p.E;
  I8Args a{};
  a.offsets = offsets;
  a.n = p.n;
  hipError_t e = launch_quantize_rows(x, 1, p.rows_max, p.d, pad64(p.d), xq, sx, rows, st);
  if (e != hipSuccess) return e;
  a.a = xq;
  a.sa = sx;
  a.b1 = (const char*)q1;
  a.b3 = (const char*)q3;
  a.s1 = s1;
  a.s3 = s3;
  a.c = h;
  a.lda = a.K = pad64(p.d);   // the bytes behind d meet zero weights
  a.N = p.f;
  a.kt = pad64(p.d) / 64;
  a.ntiles = (p.f + 15) / 16;
  if ((e = launch_product<true, false>(a, mean, all, p.T, p.rows_max, st)) != hipSuccess) return e;
  if ((e = launch_quantize_rows(h, 1, p.rows_max, p.f, pad64(p.f), hq, sh, rows, st)) != hipSuccess) return e;
  a.a = hq;
  a.sa = sh;
  a.b1 = (const char*)q2;
  a.b3 = nullptr;
  a.s1 = s2;
  a.s3 = nullptr;
  a.c = y;
  a.lda = a.K = pad64(p.f);
  a.N = p.d;
  a.kt = pad64(p.f) / 64;
  a.ntiles = (p.d + 15) / 16;
  return launch_product<false, false>(a, mean, all, p.T, p.rows_max, st);
}

}  // namespace moe
