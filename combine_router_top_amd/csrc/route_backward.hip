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

namespace moe {

constexpr int RB_TOK = 16;        // tokens of a workgroup of the logit gradients
constexpr int RB_MOST = 512;      // workgroups of it

static int rb_blocks(const Prob& p) { return (int)std::min<int64_t>(((int64_t)p.T + RB_TOK - 1) / RB_TOK, RB_MOST); }
static int rb_pad(const Prob& p) { return (p.E + 7) / 8 * 8; }

__device__ __forceinline__ float rb_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ float rb_max(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}

// Logit gradients, one wave per token, lane l holds experts l + 64 j.  dl, dlb [T][Ep]
// (either NULL): the fp32 values, those rounded to bf16 with zero columns from E on.
// colsum: this workgroup's sums over its tokens, [gridDim.x][E], or NULL.
template <int NV>
__global__ __launch_bounds__(256) void logit_grad(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                                                  const float* __restrict__ dw, int T, int E, int Ep, int k,
                                                  SelectRule r, float* __restrict__ dl, bf16_t* __restrict__ dlb,
                                                  float* __restrict__ colsum) {
  __shared__ float red[4][64 * NV];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float sum[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) sum[j] = 0.f;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < T; t += (int64_t)gridDim.x * 4) {
    float l[NV], g[NV];
    bool in[NV];
    const int my = lane < k ? idx[t * k + lane] : -1;
    const float mw = lane < k ? dw[t * k + lane] * r.scale : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane + 64 * j;
      l[j] = e < E ? logits[t * E + e] : -INFINITY;
      g[j] = 0.f;
      in[j] = false;
    }
    for (int q = 0; q < k; ++q) {
      const int e = __builtin_amdgcn_readlane(my, q);
      const float v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mw), q));
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (e == lane + 64 * j) {
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
      const float z = expf(-fabsf(l[j]));
      slope[j] = r.softmax ? 1.f : (l[j] > 0.f ? z : 1.f) / (1.f + z);   // sigmoid(-l)
      s[j] = r.softmax ? expf(l[j] - top) : expf(fminf(l[j], 0.f) - top) / (1.f + z);
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
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane + 64 * j;
      const bool live = in[j] || (r.softmax && !r.renorm);
      const float v = live ? s[j] * inv * slope[j] * (g[j] - mean) : 0.f;
      if (e < E) {
        if (dl) dl[t * E + e] = v;
        sum[j] += v;
      }
      if (dlb && e < Ep) dlb[t * Ep + e] = (bf16_t)(cvt_bf16x2(e < E ? v : 0.f, 0.f));
    }
  }
  if (!colsum) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) red[wave][lane + 64 * j] = sum[j];
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

// What remains of dWg and db: the parts' sums, in their order.
__global__ __launch_bounds__(256) void gate_sums(const float* __restrict__ part, int shares, int64_t d, int E, int Ep,
                                                 bf16_t* __restrict__ dwg, const float* __restrict__ colsum, int rows,
                                                 float* __restrict__ db) {
  if (db && blockIdx.x == 0)
    for (int e = threadIdx.x; e < E; e += 256) {
      float s = 0.f;
      for (int b = 0; b < rows; ++b) s += colsum[(int64_t)b * E + e];
      db[e] = s;
    }
  if (!dwg) return;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < d * E; i += (int64_t)gridDim.x * 256) {
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
      hipLaunchKernelGGL(gate_sums, dim3(1), dim3(256), 0, st, (const float*)nullptr, 0, (int64_t)p.d, p.E, Ep,
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
  const int64_t blocks = dwg ? std::min<int64_t>(((int64_t)p.d * p.E + 255) / 256, 4096) : 1;
  hipLaunchKernelGGL(gate_sums, dim3((unsigned)blocks), dim3(256), 0, st, (const float*)part, shares, (int64_t)p.d, p.E, Ep,
                     (bf16_t*)dwg, (const float*)colsum, rb_blocks(p), dbias);
  return hipGetLastError();
}

}  // namespace moe
