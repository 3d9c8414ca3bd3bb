// Backward pass of the router.  With l = x Wg + b, the experts S = {e_j} that a token
// chose, its scores s and the gradient g_j of its weights w_j (times `scale`, left out
// below):
//
//   sigmoid           dl_e = g_e s_e (1 - s_e)                     e in S, else 0
//   sigmoid, renorm   p = s / sum_S s,  dl_e = p_e (1 - s_e) (g_e - sum_S g p)
//   softmax           dl_e = s_e ([e in S] g_e - sum_S g s)        all e
//   softmax, renorm   p = s / sum_S s,  dl_e = p_e (g_e - sum_S g p)
//
//   dx = rnd(dx_add + rnd(dl) Wg^T)   dWg = rnd(x^T rnd(dl))   db = sum_t dl_t
//
// dl is rounded to the storage type for the two products because the matrix cores
// take it so (bf16: up to 2^-8 relative, once per value, as dg and du of the experts);
// the logit gradients that are returned and db come from the unrounded fp32 values.
#include <algorithm>

#include "common.h"
#include "f32_tile.h"
#include "kernels.h"
#include "seg_tile.h"
#include "wave_reduce.h"

namespace moe {

constexpr int RB_TOK = 4;         // tokens of a workgroup of the logit gradients
constexpr int RB_MOST = 512;      // workgroups of it

static int rb_blocks(const Prob& p) { return (int)std::min<int64_t>(((int64_t)p.T + RB_TOK - 1) / RB_TOK, RB_MOST); }
static int rb_pad(const Prob& p) { return (p.E + 7) / 8 * 8; }

__device__ __forceinline__ float rb_sum(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float rb_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

// A token's row of logit gradients, lane l with experts NV l .. NV l + NV - 1, and its sums.
template <int NV>
struct LogitRows {
  float* dl;       // [T][E] or NULL
  bf16_t* dlb;     // [T][Ep] or NULL: rounded, with zero columns from E on
  int E, Ep;
  float sum[NV];
  __device__ __forceinline__ LogitRows(float* dl, bf16_t* dlb, int E, int Ep) : dl(dl), dlb(dlb), E(E), Ep(Ep) {
#pragma unroll
    for (int j = 0; j < NV; ++j) sum[j] = 0.f;
  }
  __device__ __forceinline__ void put(int64_t t, const float (&v)[NV]) {
    const int e0 = NV * (int)(threadIdx.x & 63);
#pragma unroll
    for (int j = 0; j < NV; ++j) sum[j] += v[j];
    if (dl) {
      float* p = dl + t * E + e0;
      if (NV % 4 == 0 && E % 4 == 0 && (reinterpret_cast<uintptr_t>(dl) & 15) == 0) {
#pragma unroll
        for (int j = 0; j < NV; j += 4)
          if (e0 + j < E) *reinterpret_cast<f32x4*>(p + j) = f32x4{v[j], v[(j + 1) % NV], v[(j + 2) % NV], v[(j + 3) % NV]};
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (e0 + j < E) p[j] = v[j];
      }
    }
    if (dlb) {   // Ep is a multiple of 8
      bf16_t* p = dlb + t * Ep + e0;
      if constexpr (NV % 4 == 0) {
#pragma unroll
        for (int j = 0; j < NV; j += 4)
          if (e0 + j < Ep) *reinterpret_cast<u32x2*>(p + j) = u32x2{cvt_bf16x2(v[j], v[j + 1]), cvt_bf16x2(v[j + 2], v[j + 3])};
      } else if constexpr (NV == 2) {
        if (e0 < Ep) *reinterpret_cast<uint32_t*>(p) = cvt_bf16x2(v[0], v[1]);
      } else {
        if (e0 < Ep) p[0] = (bf16_t)cvt_bf16x2(v[0], 0.f);
      }
    }
  }
  // This workgroup's sums over its tokens: [gridDim.x][E].
  __device__ __forceinline__ void total(float* colsum, float (*red)[64 * NV]) {
    const int e0 = NV * (int)(threadIdx.x & 63);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) red[threadIdx.x >> 6][e0 + j] = sum[j];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256)
      colsum[(int64_t)blockIdx.x * E + e] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
  }
};

// Logit gradients where only the chosen experts have any: a wave per token, lane q with
// its q-th choice, whose logit is all that is read.  The row takes shape in LDS.  (Each
// lane with NV experts of the row, as below: 4096 x 256 9.7 us, so 6.1.)
template <int NV>
__global__ __launch_bounds__(256) void logit_grad_chosen(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                                                         const float* __restrict__ dw, int T, int E, int Ep, int k,
                                                         SelectRule r, float* __restrict__ dl, bf16_t* __restrict__ dlb,
                                                         float* __restrict__ colsum) {
  __shared__ float row[4][64 * NV];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e0 = NV * lane;
  LogitRows<NV> rows(dl, dlb, E, Ep);
#pragma unroll
  for (int j = 0; j < NV; ++j) row[wave][e0 + j] = 0.f;
  const int64_t step = (int64_t)gridDim.x * 4, t0 = (int64_t)blockIdx.x * 4 + wave;
  // choices two tokens ahead, the logits at them one token ahead
  auto choice = [&](int64_t t) { return t < T && lane < k ? idx[t * k + lane] : -1; };
  auto slope_of = [&](int64_t t) { return t < T && lane < k ? dw[t * k + lane] : 0.f; };
  auto logit = [&](int64_t t, int e) { return (unsigned)e < (unsigned)E ? logits[t * E + e] : -INFINITY; };
  int my = choice(t0), ni = choice(t0 + step);
  float w = slope_of(t0), nw = slope_of(t0 + step), l = logit(t0, my);
  for (int64_t t = t0; t < T; t += step) {
    const float nl = logit(t + step, ni);
    const int fi = choice(t + 2 * step);
    const float fw = slope_of(t + 2 * step), mw = w * r.scale;
    // an expert named twice counts once, with both gradients
    float g = 0.f;
    bool live = (unsigned)my < (unsigned)E;
    for (int q = 0; q < k; ++q) {
      const float v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mw), q));
      if (__builtin_amdgcn_readlane(my, q) == my) {
        g += v;
        live = live && q >= lane;
      }
    }
    const float z = expf(-fabsf(l)), part = 1.f / (1.f + z);   // sigmoid(|l|)
    const float score = r.softmax ? l : fminf(l, 0.f);
    const bool shared = r.renorm;
    const float top = shared ? rb_max(live ? score : -INFINITY) : 0.f;
    const float slope = r.softmax ? 1.f : (l > 0.f ? z : 1.f) * part;   // sigmoid(-l)
    float s = shared ? expf(score - top) * (r.softmax ? 1.f : part) : (l > 0.f ? 1.f : z) * part;
    if (!live || l == -INFINITY) s = 0.f;
    float inv = 1.f, mean = 0.f;
    if (shared) {
      const float total = rb_sum(s), dot = rb_sum(live ? g * s : 0.f);
      inv = total == 0.f ? 0.f : 1.f / total;
      mean = dot * inv;
    }
    if (live) row[wave][my] = s * inv * slope * (g - mean);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    float v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = row[wave][e0 + j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (live) row[wave][my] = 0.f;
    rows.put(t, v);
    my = ni;
    ni = fi;
    l = nl;
    w = nw;
    nw = fw;
  }
  if (colsum) rows.total(colsum, row);
}

// Logit gradients of a softmax over all experts: one wave per token, lane l holds experts
// NV l .. NV l + NV - 1.
template <int NV>
__global__ __launch_bounds__(256) void logit_grad(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                                                  const float* __restrict__ dw, int T, int E, int Ep, int k,
                                                  SelectRule r, float* __restrict__ dl, bf16_t* __restrict__ dlb,
                                                  float* __restrict__ colsum) {
  __shared__ float red[4][64 * NV];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e0 = NV * lane;
  const bool quads = NV % 4 == 0 && E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  LogitRows<NV> rows(dl, dlb, E, Ep);
  const int64_t step = (int64_t)gridDim.x * 4;
  // the next token's values are on their way while one is worked on
  float nl[NV], nw = 0.f;
  int ni = -1;
  auto load = [&](int64_t t) {
    ni = lane < k ? idx[t * k + lane] : -1;
    nw = lane < k ? dw[t * k + lane] : 0.f;
    const float* p = logits + t * E + e0;
    if (quads) {
#pragma unroll
      for (int j = 0; j < NV; j += 4) {
        f32x4 v = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (e0 + j < E) v = *reinterpret_cast<const f32x4*>(p + j);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < NV) nl[j + i] = v[i];
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) nl[j] = e0 + j < E ? p[j] : -INFINITY;
    }
  };
  int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t < T) load(t);
  for (; t < T; t += step) {
    float l[NV], g[NV];
    const int my = ni;
    const float mw = nw * r.scale;
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      l[j] = nl[j];
      g[j] = 0.f;
      top = fmaxf(top, l[j]);
    }
    if (t + step < T) load(t + step);
    for (int q = 0; q < k; ++q) {
      const int e = __builtin_amdgcn_readlane(my, q) - e0;
      const float v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mw), q));
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (e == j) g[j] += v;
    }
    top = rb_max(top);
    float s[NV], total = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      s[j] = l[j] == -INFINITY ? 0.f : expf(l[j] - top);
      total += s[j];
      dot += g[j] * s[j];
    }
    total = rb_sum(total);
    dot = rb_sum(dot);
    const float inv = total == 0.f ? 0.f : 1.f / total, mean = dot * inv;
    float v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = e0 + j < E ? s[j] * inv * (g[j] - mean) : 0.f;
    rows.put(t, v);
  }
  if (colsum) rows.total(colsum, red);
}

// Rows of Wg [d][E] at a stride of Ep, zeros between: the product's rows are read 16
// bytes at a time.
__global__ __launch_bounds__(256) void pad_rows(const bf16_t* __restrict__ w, int64_t d, int E, int Ep,
                                                bf16_t* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < d * Ep; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / Ep;
    const int e = (int)(i - row * Ep);
    out[i] = e < E ? w[row * E + e] : (bf16_t)0;
  }
}

// dx and the parts of dWg, in one launch of one workgroup per compute unit: half of the
// workgroups begin with the one, half with the other, so that what is mostly read (x)
// and what is mostly written (dx) share the memory.
//
// dx: tiles of seg_tile.h, rows of dl against rows of Wg.  K is E, a few stages, and a tile
// is mostly its store: whole rows leave through LDS, except where dx_add joins the sum
// before it is rounded, and on the small tiles of few tokens.
// dWg: a unit is 128 rows of d, 256 experts and a share of the tokens, both operands
// panels of 64 tokens in a ring of three slots, transposed by the LDS read.
// 4096 x 7168 x 256: 45 us (dx alone 26, the parts of dWg alone 23; two launches 49), at 59 MB of
// x, as much of dx and 29 MB of parts; a workgroup's stores and the loads of its next tile
// bound it, with one workgroup on a compute unit.  With dx_add the whole call takes 77 us instead
// of 54: 59 MB more, and stores in pieces of 64 bytes.
struct RouteGrad {
  const bf16_t* x;
  const bf16_t* wg;     // [d][Ep]
  const bf16_t* dl;     // [T][Ep]
  const bf16_t* add;
  bf16_t* dx;           // or NULL
  float* part;          // [shares][d][Ep], or NULL
  int T, d, Ep;
  int shares;
};

enum { RG_FEW = 0, RG_ROWS = 1, RG_ADD = 2 };   // small tiles, whole rows, with dx_add
template <int KIND>
using RowCfg = StCfg<KIND == RG_FEW ? 1 : 4, ST_ROWS, ST_ROWS, f32x4, 1, false, KIND == RG_FEW ? 2 : 16, KIND == RG_ROWS>;

// Tiles of dx.
template <int KIND>
__device__ __forceinline__ void row_tiles(const RouteGrad& p, char* ring) {
  using Cfg = RowCfg<KIND>;
  constexpr int MT = Cfg::MT;
  const int blocks = (p.T + Cfg::BM - 1) / Cfg::BM, ntn = (p.d + Cfg::BN - 1) / Cfg::BN;
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  st_run<Cfg>(
      blocks * ntn, ring,
      [&](int L, StCtx<Cfg>& c) {
        const StTile t = st_tile_of(L, 0, p.T, blocks, ntn, Cfg::BM);
        const uint32_t ld = (uint32_t)p.Ep * 2;
        st_rows(c.a[0], p.dl + (int64_t)t.r0 * p.Ep, ld, t.R, ld);
        st_rows(c.b[0], p.wg + (int64_t)Cfg::BN * t.nt * p.Ep, ld, min(Cfg::BN, p.d - Cfg::BN * t.nt), ld);
        c.nst = c.nst1 = (p.Ep + 63) / 64;
        return t;
      },
      [&](const StTile& t, typename Cfg::Acc& acc) {
        const StOut o = st_out(p.dx + (int64_t)t.r0 * p.d, (int64_t)p.d * 2, t.R);
        if constexpr (KIND == RG_ROWS) {
          store_tile_rows(o, acc, Cfg::BN * t.nt, p.d, ring + Cfg::LDS);
          return;
        }
        if (KIND == RG_FEW && !p.add) {
          st_store_tile(o, acc, Cfg::BN * t.nt, p.d);
          return;
        }
        const __amdgpu_buffer_rsrc_t ra = gc_rsrc(p.add + (int64_t)t.r0 * p.d, (uint32_t)t.R * (uint32_t)p.d * 2);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int row = 16 * MT * (wave & 3) + 16 * mt + i;
          u32x4 av[Cfg::NT / 2];
#pragma unroll
          for (int k = 0; k < Cfg::NT / 2; ++k) {
            const int col = Cfg::BN * t.nt + Cfg::WN * (wave >> 2) + 32 * k + 8 * q;
            av[k] = __builtin_amdgcn_raw_buffer_load_b128(
                ra, col < p.d ? ((uint32_t)row * (uint32_t)p.d + (uint32_t)col) * 2u : 0xFFFFFFF0u, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < Cfg::NT / 2; ++k) {
            const int col = Cfg::BN * t.nt + Cfg::WN * (wave >> 2) + 32 * k + 8 * q;
            float x[4], y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              x[r] = acc[mt][2 * k][r];
              y[r] = acc[mt][2 * k + 1][r];
              st_swap_pair(x[r], y[r]);   // x: columns 8 q + r, y: 8 q + 4 + r
            }
            u32x4 v;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const float* z = h < 2 ? x + 2 * h : y + 2 * (h - 2);
              v[h] = cvt_bf16x2(z[0] + bf16_lo(av[k][h]), z[1] + bf16_hi(av[k][h]));
            }
            st_put(o, row, 2u * (uint32_t)col, col < p.d, v);
          }
        }
      });
}

constexpr int RG_XB = 64 * 256, RG_SLOT = 3 * RG_XB;   // a stage's 64 x 128 of x, with 64 x 256 of dl
constexpr int RG_LDS = 3 * RG_SLOT;

__device__ __forceinline__ void weight_unit(const RouteGrad& p, int u, char* lds) {
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int nn = (p.Ep + 255) / 256, stages = (p.T + 63) / 64, each = (stages + p.shares - 1) / p.shares;
  // the shares of a block of rows run far apart, neighbours share their dl in an L2
  const int md = st_div(u, nn * p.shares), rest = u - md * nn * p.shares, share = st_div(rest, nn), nb = rest - share * nn;
  const int64_t first = (int64_t)64 * each * share;
  const int rows = __builtin_amdgcn_readfirstlane((int)max((int64_t)0, min((int64_t)p.T - first, (int64_t)64 * each)));
  const int nst = (rows + 63) / 64;
  const uint32_t lbase = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(dt_lds_t*)lds);
  // x: copy c of wave w holds K-rows 8 w + 4 c .. + 3 of the half-panel
  const uint32_t ldx = (uint32_t)p.d * 2u;
  const int sig = (lane >> 4) | ((wave & 1) << 2);
  const int xcol = 128 * md + 8 * ((lane & 15) ^ (2 * sig));
  const uint32_t vx = xcol < p.d ? (uint32_t)(8 * wave + (lane >> 4)) * ldx + 2u * (uint32_t)xcol : GC_OOR;
  const char* xb = (const char*)(p.x + first * p.d);
  StOp<ST_PANEL, 256> q;
  st_panel(q, p.dl + first * p.Ep, (uint32_t)p.Ep * 2u, rows, 256 * nb, p.Ep);
  auto issue = [&](int slot, int st) {
    const uint32_t at = lbase + slot * RG_SLOT;
    const int left = __builtin_amdgcn_readfirstlane(max(0, min(64, rows - 64 * st)));
    const __amdgpu_buffer_rsrc_t r = gc_rsrc(xb + (int64_t)st * 64 * ldx, (uint32_t)left * ldx);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      bd_copy16(r, at + 2048 * wave + 1024 * c, vx, st_offset((uint32_t)(4 * c) * ldx, (uint32_t)left * ldx));
    st_issue(q, at + RG_XB, st);
  };
  f32x4 acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[a][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int xo = st_lane<ST_PANEL>(4 * wm), lo = st_lane<ST_PANEL>(4 * wn);
  if (nst > 0) issue(0, 0);
  if (nst > 1) issue(1, 1);
  int slot = 0;
  for (int s = 0; s < nst; ++s) {
    // this stage has arrived in every wave, all are done with the one before
    if (s + 1 < nst) st_sync<6>();
    else st_sync<0>();
    const int third = slot == 0 ? 2 : slot - 1;
    if (s + 2 < nst) issue(third, s + 2);
    const char* at = lds + slot * RG_SLOT;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4 xf[4], lf[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        xf[t] = st_frag<ST_PANEL>(at, xo, ks, t);
        lf[t] = st_frag<ST_PANEL>(at + RG_XB, lo, ks, t);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) acc[mt][t] = st_mfma(lf[t], xf[mt], acc[mt][t]);
    }
    slot = slot == 2 ? 0 : slot + 1;
  }
  const int row0 = 128 * md;
  const StOut o = st_out(p.part + ((int64_t)share * p.d + row0) * p.Ep, (int64_t)p.Ep * 4, min(128, p.d - row0));
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int col = 256 * nb + 64 * wn + 16 * t + 4 * g;
      st_put(o, 64 * wm + 16 * mt + i, 4u * (uint32_t)col, col < p.Ep, __builtin_bit_cast(u32x4, acc[mt][t]));
    }
  __syncthreads();   // before LDS is written again
}

template <int KIND>
__global__ __launch_bounds__(512, 1) void route_grad(RouteGrad p) {
  constexpr int LR = RowCfg<KIND>::LDS + (KIND == RG_ROWS ? 8 * 4096 : 0);
  __shared__ __attribute__((aligned(16))) char lds[LR > RG_LDS ? LR : RG_LDS];
  for (int phase = 0; phase < 2; ++phase) {
    if ((((int)blockIdx.x >> 3) + phase) & 1) {
      if (p.dx) row_tiles<KIND>(p, lds);
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");   // all are done with LDS
    } else if (p.part) {
      const int units = (p.d + 127) / 128 * ((p.Ep + 255) / 256) * p.shares;
      // from the other end, so that a workgroup with a tile less of dx has a unit more
      for (int u = (int)gridDim.x - 1 - st_first_tile(); u < units; u += (int)gridDim.x) weight_unit(p, u, lds);
    }
  }
}

// 64 values of db, from expert 64 * block on, by NW waves: the rows of colsum dealt out over
// sixteen sums, whatever NW is, sixteen loads together.
template <int NW>
__device__ __forceinline__ void bias_sums(const float* colsum, int rows, int E, int block, float* db, float (*red)[64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = 64 * block + lane;
  float s;
  for (int w = wave; w < 16; w += NW) {
    s = 0.f;
    for (int b = w; b < rows; b += 256) {
      float v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) v[u] = e < E && b + 16 * u < rows ? colsum[(int64_t)(b + 16 * u) * E + e] : 0.f;
#pragma unroll
      for (int u = 0; u < 16; ++u) s += v[u];
    }
    red[w][lane] = s;
  }
  __syncthreads();
  if (wave == 0 && e < E) {
    s = red[0][lane];
    for (int u = 1; u < 16; ++u) s += red[u][lane];
    db[e] = s;
  }
}

// What remains of dWg and db, the parts' sums in their order.  The first ceil(E / 64)
// workgroups sum db if it is wanted.  (4096 x 7168 x 256: 6.3 us, 29 MB of parts from the caches.)
__global__ __launch_bounds__(1024) void gate_sums(const float* __restrict__ part, int shares, int64_t d, int E, int Ep,
                                                  bf16_t* __restrict__ dwg, const float* __restrict__ colsum, int rows,
                                                  float* __restrict__ db) {
  __shared__ float red[16][64];
  int first = 0;
  if (db) {
    first = (E + 63) / 64;
    if ((int)blockIdx.x < first) {
      bias_sums<16>(colsum, rows, E, blockIdx.x, db, red);
      return;
    }
  }
  const int64_t at0 = ((int64_t)blockIdx.x - first) * 1024 + threadIdx.x, step = ((int64_t)gridDim.x - first) * 1024;
  if (E == Ep) {   // 8 values of a row together
    for (int64_t i = at0; i < d * E / 8; i += step) {
      f32x4 a = f32x4{0.f, 0.f, 0.f, 0.f}, b = a;
      for (int q = 0; q < shares; ++q) {
        const f32x4* v = reinterpret_cast<const f32x4*>(part + q * d * Ep) + 2 * i;
        a += v[0];
        b += v[1];
      }
      reinterpret_cast<u32x4*>(dwg)[i] =
          u32x4{cvt_bf16x2(a[0], a[1]), cvt_bf16x2(a[2], a[3]), cvt_bf16x2(b[0], b[1]), cvt_bf16x2(b[2], b[3])};
    }
    return;
  }
  for (int64_t i = at0; i < d * E; i += step) {
    const int64_t row = i / E, at = row * Ep + (i - row * E);
    float s = 0.f;
    for (int q = 0; q < shares; ++q) s += part[q * d * Ep + at];
    dwg[i] = (bf16_t)cvt_bf16x2(s, 0.f);
  }
}

// fp32: 32 x 32 tiles of dx (the first in_tiles workgroups) and of dWg; then db, 64 values a
// workgroup (64 x 128 x 8: a launch of its own for db 2.2 us more).
struct RouteGradF32 {
  const float* dl;
  const float* x;
  const float* wg;
  const float* add;
  float* dx;
  float* dwg;
  int T, d, E;
  int64_t in_tiles, tiles;
  const float* colsum;
  int rows;
  float* db;   // or NULL
};
__global__ __launch_bounds__(64 * F_NW) void route_grad_f32(RouteGradF32 p) {
  __shared__ __attribute__((aligned(16))) F32Lds s;
  int64_t tile = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (tile >= p.tiles) {
    const int64_t block = tile - p.tiles;
    if (p.db && block < (p.E + 63) / 64) bias_sums<F_NW>(p.colsum, p.rows, p.E, (int)block, p.db, reinterpret_cast<float(*)[64]>(&s));
    return;
  }
  const int nd = (p.d + F_T - 1) / F_T, ne = (p.E + F_T - 1) / F_T;
  float acc[4][4] = {};
  if (tile < p.in_tiles) {
    const int64_t r0 = tile / nd * F_T;
    const int c0 = (int)(tile % nd) * F_T, R = (int)min((int64_t)F_T, (int64_t)p.T - r0);
    const float* a = p.dl + r0 * p.E;
    const float* b = p.wg + (int64_t)c0 * p.E;
    f32_tile([&](int k, int j) { return j < R ? a[(int64_t)j * p.E + k] : 0.f; }, true,
             [&](int k, int j) { return c0 + j < p.d ? b[(int64_t)j * p.E + k] : 0.f; }, true, p.E, s, acc);
    f32x2 v = f32_join(s, acc);
    const int row = f32_row(), col = c0 + f32_col();
    if (row >= R || col >= p.d) return;
    const int64_t at = (r0 + row) * p.d + col;
    if (p.add) v += *reinterpret_cast<const f32x2*>(p.add + at);
    *reinterpret_cast<f32x2*>(p.dx + at) = v;
  } else {
    tile -= p.in_tiles;
    const int m0 = (int)(tile / ne) * F_T, n0 = (int)(tile % ne) * F_T;
    f32_tile([&](int k, int j) { return m0 + j < p.d ? p.x[(int64_t)k * p.d + m0 + j] : 0.f; }, false,
             [&](int k, int j) { return n0 + j < p.E ? p.dl[(int64_t)k * p.E + n0 + j] : 0.f; }, false, p.T, s, acc);
    const f32x2 v = f32_join(s, acc);
    const int row = m0 + f32_row(), col = n0 + f32_col();
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (row < p.d && col + r < p.E) p.dwg[(int64_t)row * p.E + col + r] = v[r];
  }
}

__global__ __launch_bounds__(256) void clear_grads(char* __restrict__ a, int64_t bytes, float* __restrict__ b, int n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < bytes / 2; i += (int64_t)gridDim.x * 256)
    reinterpret_cast<uint16_t*>(a)[i] = 0;
  if (b && blockIdx.x == 0)
    for (int i = threadIdx.x; i < n; i += 256) b[i] = 0.f;
}

static size_t pad256(size_t v) { return (v + 255) / 256 * 256; }

static int rb_shares(const Prob& p) { return route_shares(device_cus(), p.T, p.d, p.E); }

struct RouteBackWs {
  size_t dl, wg, part, colsum, total;
};
static RouteBackWs rb_ws(const Prob& p) {
  RouteBackWs w;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += pad256(bytes);
    return at;
  };
  w.dl = take((size_t)p.T * (p.dtype == 1 ? 2 * rb_pad(p) : 4 * p.E));
  w.wg = take(p.dtype == 1 && p.E % 8 ? (size_t)p.d * rb_pad(p) * 2 : 0);
  w.part = take(p.dtype == 1 ? (size_t)rb_shares(p) * p.d * rb_pad(p) * 4 : 0);
  w.colsum = take((size_t)rb_blocks(p) * p.E * 4);
  w.total = o;
  return w;
}
size_t route_backward_ws_bytes(const Prob& p) { return rb_ws(p).total; }

hipError_t launch_route_backward(const Prob& p, const SelectRule& r, const void* x, const void* wg, const float* logits,
                                 const int32_t* idx, const float* dw, const void* dx_add, float* dlogits, void* dx,
                                 void* dwg, float* dbias, void* ws, hipStream_t st) {
  hipError_t e;
  if (p.T == 0) {
    const int64_t bytes = dwg ? (int64_t)p.d * p.E * p.elem() : 0;
    if (!dwg && !dbias) return hipSuccess;
    hipLaunchKernelGGL(clear_grads, dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(bytes / 512, 2048))), dim3(256), 0,
                       st, (char*)dwg, bytes, dbias, p.E);
    return hipGetLastError();
  }
  const RouteBackWs L = rb_ws(p);
  char* at = (char*)ws;
  const bool products = dx || dwg;
  const int Ep = p.dtype == 1 ? rb_pad(p) : p.E;
  bf16_t* dlb = p.dtype == 1 && products ? (bf16_t*)(at + L.dl) : nullptr;
  float* dl = dlogits ? dlogits : p.dtype == 1 || !products ? nullptr : (float*)(at + L.dl);
  float* colsum = dbias ? (float*)(at + L.colsum) : nullptr;
  const int nv = (p.E + 63) / 64;
  auto all = nv <= 1 ? logit_grad<1> : nv <= 2 ? logit_grad<2> : nv <= 4 ? logit_grad<4> : nv <= 8 ? logit_grad<8> : logit_grad<16>;
  auto chosen = nv <= 1   ? logit_grad_chosen<1>
                : nv <= 2 ? logit_grad_chosen<2>
                : nv <= 4 ? logit_grad_chosen<4>
                : nv <= 8 ? logit_grad_chosen<8>
                          : logit_grad_chosen<16>;
  hipLaunchKernelGGL(r.softmax && !r.renorm ? all : chosen, dim3((unsigned)rb_blocks(p)), dim3(256), 0, st, logits, idx, dw, p.T, p.E, Ep, p.k, r, dl, dlb,
                     colsum);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (p.dtype != 1) {
    if (products) {
      RouteGradF32 q{dl, (const float*)x, (const float*)wg, (const float*)dx_add, (float*)dx, (float*)dwg, p.T, p.d, p.E};
      const int64_t nd = (p.d + F_T - 1) / F_T, ne = (p.E + F_T - 1) / F_T;
      q.in_tiles = dx ? ((int64_t)p.T + F_T - 1) / F_T * nd : 0;
      q.tiles = q.in_tiles + (dwg ? nd * ne : 0);
      q.colsum = colsum;
      q.rows = rb_blocks(p);
      q.db = dbias;
      const int64_t all = q.tiles + (dbias ? (p.E + 63) / 64 : 0), gx = std::min<int64_t>(all, 1 << 16);
      hipLaunchKernelGGL(route_grad_f32, dim3((unsigned)gx, (unsigned)((all + gx - 1) / gx)), dim3(64 * F_NW), 0, st, q);
    } else if (dbias) {
      hipLaunchKernelGGL(gate_sums, dim3((unsigned)((p.E + 63) / 64)), dim3(1024), 0, st, (const float*)nullptr, 0, (int64_t)p.d, p.E, Ep,
                         (bf16_t*)nullptr, (const float*)colsum, rb_blocks(p), dbias);
    }
    return hipGetLastError();
  }
  if (!products && !dbias) return hipSuccess;
  const int shares = rb_shares(p);
  float* part = (float*)(at + L.part);
  if (products) {
    const bf16_t* w = (const bf16_t*)wg;
    if (dx && p.E % 8) {
      w = (const bf16_t*)(at + L.wg);
      hipLaunchKernelGGL(pad_rows, dim3((unsigned)std::min<int64_t>(((int64_t)p.d * Ep + 255) / 256, 4096)), dim3(256), 0, st,
                         (const bf16_t*)wg, (int64_t)p.d, p.E, Ep, (bf16_t*)(at + L.wg));
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    RouteGrad q{(const bf16_t*)x, w, dlb, (const bf16_t*)dx_add, (bf16_t*)dx, dwg ? part : nullptr, p.T, p.d, Ep, shares};
    const int64_t tiles = (((int64_t)p.T + 255) / 256) * ((p.d + 255) / 256);
    const bool few = route_few(device_cus(), p.T, p.d);
    int64_t units = dwg ? (int64_t)((p.d + 127) / 128) * ((Ep + 255) / 256) * shares : 0;
    if (dx) units += few ? (((int64_t)p.T + 63) / 64) * ((p.d + 127) / 128) : tiles;
    auto kern = few ? route_grad<RG_FEW> : dx_add ? route_grad<RG_ADD> : route_grad<RG_ROWS>;
    hipLaunchKernelGGL(kern, dim3(st_grid(units)), dim3(512), 0, st, q);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (!dwg && !dbias) return hipSuccess;
  const int64_t count = !dwg ? 0 : p.E == Ep ? (int64_t)p.d * p.E / 8 : (int64_t)p.d * p.E;
  const int64_t blocks = std::min<int64_t>((count + 1023) / 1024, 1024) + (dbias ? (p.E + 63) / 64 : 0);
  hipLaunchKernelGGL(gate_sums, dim3((unsigned)blocks), dim3(1024), 0, st, (const float*)part, shares, (int64_t)p.d, p.E, Ep,
                     (bf16_t*)dwg, (const float*)colsum, rb_blocks(p), dbias);
  return hipGetLastError();
}

}  // namespace moe
