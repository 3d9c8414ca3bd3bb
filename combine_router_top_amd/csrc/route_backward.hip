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

constexpr int RB_TOK = 8;         // tokens of a workgroup of the logit gradients
constexpr int RB_MOST = 512;      // workgroups of it

static int rb_blocks(const Prob& p) { return (int)std::min<int64_t>(((int64_t)p.T + RB_TOK - 1) / RB_TOK, RB_MOST); }
static int rb_pad(const Prob& p) { return (p.E + 7) / 8 * 8; }

__device__ __forceinline__ float rb_sum(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float rb_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

// Logit gradients, one wave per token, lane l holds experts NV l .. NV l + NV - 1.  dl
// [T][E], dlb [T][Ep] (either NULL): the fp32 values, those rounded to bf16 with zero
// columns from E on.  colsum: this workgroup's sums over its tokens, [gridDim.x][E], or NULL.
template <int NV>
__global__ __launch_bounds__(256) void logit_grad(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                                                  const float* __restrict__ dw, int T, int E, int Ep, int k,
                                                  SelectRule r, float* __restrict__ dl, bf16_t* __restrict__ dlb,
                                                  float* __restrict__ colsum) {
  __shared__ float red[4][64 * NV];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e0 = NV * lane;
  const bool quads = NV % 4 == 0 && E % 4 == 0 && ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dl)) & 15) == 0;
  float sum[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) sum[j] = 0.f;
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
    bool in[NV];
    const int my = ni;
    const float mw = nw * r.scale;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      l[j] = nl[j];
      g[j] = 0.f;
      in[j] = false;
    }
    if (t + step < T) load(t + step);
    for (int q = 0; q < k; ++q) {
      const int e = __builtin_amdgcn_readlane(my, q) - e0;
      const float v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mw), q));
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (e == j) {
          g[j] += v;
          in[j] = true;
        }
    }
    // scores up to a common factor (the sum over all experts, or over the chosen
    // ones), and what the slope of a score holds beside it
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float v = r.softmax ? l[j] : fminf(l[j], 0.f);
      if (!r.renorm || in[j]) top = fmaxf(top, v);
    }
    top = r.softmax || r.renorm ? rb_max(top) : 0.f;
    float s[NV], slope[NV], total = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (r.softmax) {
        slope[j] = 1.f;
        s[j] = expf(l[j] - top);
      } else {
        const float z = expf(-fabsf(l[j])), inv = 1.f / (1.f + z);
        slope[j] = (l[j] > 0.f ? z : 1.f) * inv;   // sigmoid(-l)
        s[j] = r.renorm ? expf(fminf(l[j], 0.f) - top) * inv : (l[j] > 0.f ? 1.f : z) * inv;
      }
      if (l[j] == -INFINITY) s[j] = 0.f;
      if (!r.renorm || in[j]) total += s[j];
      dot += g[j] * s[j];
    }
    const bool shared = r.softmax || r.renorm;
    if (shared) {
      total = rb_sum(total);
      dot = rb_sum(dot);
    }
    const float inv = !shared ? 1.f : total == 0.f ? 0.f : 1.f / total;
    const float mean = shared ? dot * inv : 0.f;
    float v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool live = e0 + j < E && (in[j] || (r.softmax && !r.renorm));
      v[j] = live ? s[j] * inv * slope[j] * (g[j] - mean) : 0.f;
      sum[j] += v[j];
    }
    if (dl) {
      float* p = dl + t * E + e0;
      if (quads) {
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
  if (!colsum) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) red[wave][e0 + j] = sum[j];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256)
    colsum[(int64_t)blockIdx.x * E + e] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
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

template <int MT>
using RowCfg = StCfg<MT, ST_ROWS, ST_ROWS, f32x4, 1, false, (MT == 1 ? 2 : 4) * MT>;

// dx tiles: rows of dl against rows of Wg.
template <int MT>
__global__ __launch_bounds__(ST_NT, 1) void row_grad(const bf16_t* __restrict__ dl, const bf16_t* __restrict__ wg,
                                                     const bf16_t* add, bf16_t* dx, int T,
                                                     int d, int Ep, int ntn) {
  using Cfg = RowCfg<MT>;
  __shared__ __attribute__((aligned(16))) char ring[Cfg::LDS];
  const int blocks = (T + Cfg::BM - 1) / Cfg::BM;
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  st_run<Cfg>(
      blocks * ntn, ring,
      [&](int L, StCtx<Cfg>& c) {
        const StTile t = st_tile_of(L, 0, T, blocks, ntn, Cfg::BM);
        const uint32_t ld = (uint32_t)Ep * 2;
        st_rows(c.a[0], dl + (int64_t)t.r0 * Ep, ld, t.R, ld);
        st_rows(c.b[0], wg + (int64_t)Cfg::BN * t.nt * Ep, ld, min(Cfg::BN, d - Cfg::BN * t.nt), ld);
        c.nst = c.nst1 = (Ep + 63) / 64;
        return t;
      },
      [&](const StTile& t, typename Cfg::Acc& acc) {
        const StOut o = st_out(dx + (int64_t)t.r0 * d, (int64_t)d * 2, t.R);
        if (!add) {
          st_store_tile(o, acc, Cfg::BN * t.nt, d);
          return;
        }
        const __amdgpu_buffer_rsrc_t ra = gc_rsrc(add + (int64_t)t.r0 * d, (uint32_t)t.R * (uint32_t)d * 2);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int row = 16 * MT * (wave & 3) + 16 * mt + i;
          u32x4 av[Cfg::NT / 2];
#pragma unroll
          for (int k = 0; k < Cfg::NT / 2; ++k) {
            const int col = Cfg::BN * t.nt + Cfg::WN * (wave >> 2) + 32 * k + 8 * q;
            av[k] = __builtin_amdgcn_raw_buffer_load_b128(
                ra, col < d ? ((uint32_t)row * (uint32_t)d + (uint32_t)col) * 2u : 0xFFFFFFF0u, 0, 0);
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
            st_put(o, row, 2u * (uint32_t)col, col < d, v);
          }
        }
      });
}

using GateWCfg = StCfg<4, ST_PANEL, ST_PANEL, f32x4, 1, false, 32>;

// Parts of dWg: tile (256 rows of d) x (256 experts) over an equal share of the
// tokens, fp32 sums at part[share][d][Ep].
__global__ __launch_bounds__(ST_NT, 1) void gate_weight_grad(const bf16_t* __restrict__ x,
                                                             const bf16_t* __restrict__ dl, float* __restrict__ part,
                                                             int T, int d, int Ep, int shares) {
  using Cfg = GateWCfg;
  __shared__ __attribute__((aligned(16))) char ring[Cfg::LDS];
  const int nm = (d + 255) / 256, nn = (Ep + 255) / 256;
  const int stages = (T + 63) / 64, each = (stages + shares - 1) / shares;
  struct Unit {
    int m, n, s, rows, nst;
  };
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  st_run<Cfg>(
      nm * nn * shares, ring,
      [&](int L, StCtx<Cfg>& c) {
        Unit u;
        u.s = st_div(L, nm * nn);
        const int at = L - u.s * nm * nn;
        u.m = st_div(at, nn);
        u.n = at - u.m * nn;
        const int64_t first = (int64_t)64 * each * u.s;
        u.rows = (int)max((int64_t)0, min((int64_t)T - first, (int64_t)64 * each));
        u.rows = __builtin_amdgcn_readfirstlane(u.rows);
        st_panel(c.a[0], x + first * d, (uint32_t)d * 2, u.rows, 256 * u.m, d);
        st_panel(c.b[0], dl + first * Ep, (uint32_t)Ep * 2, u.rows, 256 * u.n, Ep);
        c.nst = c.nst1 = u.nst = (u.rows + 63) / 64;
        return u;
      },
      [&](const Unit& u, typename Cfg::Acc& acc) {
        const int row0 = 256 * u.m;
        const StOut o = st_out(part + ((int64_t)u.s * d + row0) * Ep, (int64_t)Ep * 4, min(256, d - row0));
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const int col = 256 * u.n + 128 * (wave >> 2) + 16 * t + 4 * (lane >> 4);
            st_put(o, 64 * (wave & 3) + 16 * mt + (lane & 15), 4u * (uint32_t)col, col < Ep,
                   __builtin_bit_cast(u32x4, acc[mt][t]));
          }
      });
}

// What remains of dWg and db, the parts' sums in their order.  The first ceil(E / 64)
// workgroups sum db if it is wanted: 64 experts, the rows dealt out over 16 waves.
__global__ __launch_bounds__(1024) void gate_sums(const float* __restrict__ part, int shares, int64_t d, int E, int Ep,
                                                  bf16_t* __restrict__ dwg, const float* __restrict__ colsum, int rows,
                                                  float* __restrict__ db) {
  __shared__ float red[16][64];
  int first = 0;
  if (db) {
    first = (E + 63) / 64;
    if ((int)blockIdx.x < first) {
      const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = 64 * blockIdx.x + lane;
      float s = 0.f;
      for (int b = wave; b < rows; b += 256) {   // sixteen loads together
        float v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) v[u] = e < E && b + 16 * u < rows ? colsum[(int64_t)(b + 16 * u) * E + e] : 0.f;
#pragma unroll
        for (int u = 0; u < 16; ++u) s += v[u];
      }
      red[wave][lane] = s;
      __syncthreads();
      if (wave == 0 && e < E) {
        s = red[0][lane];
        for (int u = 1; u < 16; ++u) s += red[u][lane];
        db[e] = s;
      }
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

// fp32: 32 x 32 tiles of dx (the first in_tiles workgroups) and of dWg.
struct RouteGradF32 {
  const float* dl;
  const float* x;
  const float* wg;
  const float* add;
  float* dx;
  float* dwg;
  int T, d, E;
  int64_t in_tiles, tiles;
};
__global__ __launch_bounds__(64 * F_NW) void route_grad_f32(RouteGradF32 p) {
  __shared__ __attribute__((aligned(16))) F32Lds s;
  int64_t tile = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (tile >= p.tiles) return;
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

// Shares of the tokens that the tiles of dWg are split into: as many as give every
// compute unit one, each of at least four stages.
static int rb_shares(const Prob& p) {
  const int64_t tiles = (int64_t)((p.d + 255) / 256) * ((p.E + 255) / 256), stages = ((int64_t)p.T + 63) / 64;
  return (int)std::max<int64_t>(1, std::min<int64_t>(device_cus() / tiles, stages / 4));
}

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
  auto kern = nv <= 1 ? logit_grad<1> : nv <= 2 ? logit_grad<2> : nv <= 4 ? logit_grad<4> : nv <= 8 ? logit_grad<8> : logit_grad<16>;
  hipLaunchKernelGGL(kern, dim3((unsigned)rb_blocks(p)), dim3(256), 0, st, logits, idx, dw, p.T, p.E, Ep, p.k, r, dl, dlb,
                     colsum);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (p.dtype != 1) {
    if (products) {
      RouteGradF32 q{dl, (const float*)x, (const float*)wg, (const float*)dx_add, (float*)dx, (float*)dwg, p.T, p.d, p.E};
      const int64_t nd = (p.d + F_T - 1) / F_T, ne = (p.E + F_T - 1) / F_T;
      q.in_tiles = dx ? ((int64_t)p.T + F_T - 1) / F_T * nd : 0;
      q.tiles = q.in_tiles + (dwg ? nd * ne : 0);
      const int64_t gx = std::min<int64_t>(q.tiles, 1 << 16);
      hipLaunchKernelGGL(route_grad_f32, dim3((unsigned)gx, (unsigned)((q.tiles + gx - 1) / gx)), dim3(64 * F_NW), 0, st, q);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (dbias)
      hipLaunchKernelGGL(gate_sums, dim3((unsigned)((p.E + 63) / 64)), dim3(1024), 0, st, (const float*)nullptr, 0, (int64_t)p.d, p.E, Ep,
                         (bf16_t*)nullptr, (const float*)colsum, rb_blocks(p), dbias);
    return hipGetLastError();
  }
  if (dx) {
    const bf16_t* w = (const bf16_t*)wg;
    if (p.E % 8) {
      w = (const bf16_t*)(at + L.wg);
      hipLaunchKernelGGL(pad_rows, dim3((unsigned)std::min<int64_t>(((int64_t)p.d * Ep + 255) / 256, 4096)), dim3(256), 0, st,
                         (const bf16_t*)wg, (int64_t)p.d, p.E, Ep, (bf16_t*)(at + L.wg));
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    e = st_with_height(st_height(device_cus(), 1, p.T, (int64_t)Ep * 2, p.d, 128), [&](auto h) {
      constexpr int bn = RowCfg<h()>::BN;
      const int ntn = (p.d + bn - 1) / bn;
      hipLaunchKernelGGL(row_grad<h()>, st_row_grid(p.T, 1, h(), ntn), dim3(ST_NT), 0, st, (const bf16_t*)dlb, w,
                         (const bf16_t*)dx_add, (bf16_t*)dx, p.T, p.d, Ep, ntn);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (!dwg && !dbias) return hipSuccess;
  const int shares = rb_shares(p);
  float* part = (float*)(at + L.part);
  if (dwg) {
    const int64_t tiles = (int64_t)((p.d + 255) / 256) * ((Ep + 255) / 256) * shares;
    hipLaunchKernelGGL(gate_weight_grad, dim3(st_grid(tiles)), dim3(ST_NT), 0, st, (const bf16_t*)x, (const bf16_t*)dlb,
                       part, p.T, p.d, Ep, shares);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const int64_t count = !dwg ? 0 : p.E == Ep ? (int64_t)p.d * p.E / 8 : (int64_t)p.d * p.E;
  const int64_t blocks = std::min<int64_t>((count + 1023) / 1024, 1024) + (dbias ? (p.E + 63) / 64 : 0);
  hipLaunchKernelGGL(gate_sums, dim3((unsigned)blocks), dim3(1024), 0, st, (const float*)part, shares, (int64_t)p.d, p.E, Ep,
                     (bf16_t*)dwg, (const float*)colsum, rb_blocks(p), dbias);
  return hipGetLastError();
}

}  // namespace moe
