// Choice of experts from router logits, with softmax or sigmoid scores, a bias for
// balance, groups of experts and weights that are renormalised or not.  For a
// token with logits l and scores s = sigmoid(l) or softmax(l) over all E experts:
//
//   c_e  = s_e + balance_e          (the value experts are chosen by)
//   groups of E / groups neighbouring experts: a group's value is the sum of its
//          group_top (1 or 2) largest c; the topk_groups best groups stay
//   idx  = the k largest c within them, descending, ties to the lower index
//   w_j  = scale s_j, or scale s_j / sum_i<k s_i (renorm)
//
// Softmax scores without a bias order experts as their logits do, and are ordered by
// them.  An expert whose logit or bias is -inf comes after every other one of its
// group.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

// Below every value that can be chosen by (scores lie in [0, 1], biases are finite).
constexpr double SEL_LOW = -1e300;

__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t u = __double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

template <class T>
__device__ __forceinline__ T wave_max_of(T v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = max(v, __shfl_xor(v, off));
  return v;
}
template <class T>
__device__ __forceinline__ T wave_sum_of(T v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// A value that is no number, or below, is the lowest.
__device__ __forceinline__ double sel_floor(double c) { return c >= SEL_LOW ? c : SEL_LOW; }

// Groups that stay, as a mask with bit g (64 / groups rounded down to a power of two)
// of each.  L lanes work on a group: lane g L + r on its members r, r + L, ..
__device__ __forceinline__ uint64_t open_groups(const double* value, int E, const SelectRule& r) {
  const int lane = threadIdx.x & 63, L = r.lanes, g = lane / L, per = E / r.groups;
  double a = -INFINITY, b = -INFINITY;   // the two largest
  if (g < r.groups)
    for (int i = lane % L; i < per; i += L) {
      const double v = value[g * per + i];
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
    }
  for (int off = 1; off < L; off <<= 1) {
    const double x = __shfl_xor(a, off), y = __shfl_xor(b, off);
    b = fmax(fmin(a, x), fmax(b, y));
    a = fmax(a, x);
  }
  const double mine = r.group_top == 2 ? a + b : a;
  int better = 0;
  for (int q = 0; q < r.groups; ++q) {
    const double v = __shfl(mine, q * L);
    better += v > mine || (v == mine && q < g);
  }
  return __ballot(g < r.groups && better < r.topk_groups);
}

// One wave per token.  NV = values per lane; lane l holds experts l + 64 j.
template <int NV>
__global__ __launch_bounds__(256) void select_kernel(const float* __restrict__ part, int nsplit,
                                                     const float* __restrict__ bias,
                                                     const float* __restrict__ balance,
                                                     float* __restrict__ logits_out, int T, int E, int k, SelectRule r,
                                                     int32_t* __restrict__ idx, float* __restrict__ w) {
  __shared__ double value[4][64 * NV];
  __shared__ float logit[4][64 * NV];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t sstride = (int64_t)T * E;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < T; t += (int64_t)gridDim.x * 4) {
    const float* pt = part + t * E;
    float l[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane + 64 * j;
      l[j] = -INFINITY;
      if (e >= E) continue;
      float v = pt[e];
      for (int s = 1; s < nsplit; ++s) v += pt[s * sstride + e];
      if (bias) v += bias[e];
      if (logits_out) logits_out[t * E + e] = v;
      l[j] = v;
      logit[wave][e] = v;
    }
    float top = l[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) top = fmaxf(top, l[j]);
    top = wave_max_of(top);
    double total = 1.0;
    double c[NV];
    if (r.softmax) {
      total = 0.0;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = lane + 64 * j;
        c[j] = e < E ? exp((double)l[j] - (double)top) : 0.0;
        total += c[j];
      }
      total = wave_sum_of(total);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) c[j] = 1.0 / (1.0 + exp(-(double)l[j]));
    }
    if (r.groups > 1 || !r.by_logit) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = lane + 64 * j;
        c[j] /= total;
        if (balance && e < E) c[j] += (double)balance[e];
        c[j] = l[j] == -INFINITY ? SEL_LOW : sel_floor(c[j]);
        if (r.groups > 1 && e < E) value[wave][e] = c[j];
      }
    }
    if (r.by_logit) {
#pragma unroll
      for (int j = 0; j < NV; ++j) c[j] = sel_floor((double)l[j]);
    }
    lds_wave_order();
    uint64_t key[NV];
    const uint64_t open = r.groups > 1 ? open_groups(value[wave], E, r) : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane + 64 * j;
      const bool in = e < E && (r.groups == 1 || ((open >> (e / (E / r.groups) * r.lanes)) & 1));
      key[j] = in ? order_key(c[j]) : 0;
    }
    int mye = 0;
    for (int q = 0; q < k; ++q) {
      uint64_t best = key[0];
      int bj = 0;
#pragma unroll
      for (int j = 1; j < NV; ++j)
        if (key[j] > best) {
          best = key[j];
          bj = j;
        }
      const uint64_t m = wave_max_of(best);
      int e = best == m ? lane + 64 * bj : 0x7FFFFFFF;
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) e = min(e, __shfl_xor(e, off));
      if (lane == q) mye = e;
      if ((e & 63) == lane) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (j == (e >> 6)) key[j] = 0;
      }
    }
    double s = 0.0;
    if (lane < k) {
      const double v = logit[wave][mye];
      s = r.softmax ? exp(v - (double)top) / total : 1.0 / (1.0 + exp(-v));
      if (logit[wave][mye] == -INFINITY && top == -INFINITY) s = 0.0;   // every logit is -inf
    }
    if (r.renorm) {
      const double sum = wave_sum_of(s);
      s = sum == 0.0 ? 0.0 : s / sum;
    }
    if (lane < k) {
      idx[t * k + lane] = mye;
      w[t * k + lane] = (float)(s * (double)r.scale);
    }
    lds_wave_order();
  }
}

hipError_t launch_select(const Prob& p, const SelectRule& r, const float* part, int nsplit, const float* bias,
                         const float* balance, float* logits, int32_t* idx, float* w, hipStream_t st) {
  const int nv = (p.E + 63) / 64;
  auto kern = nv <= 1   ? select_kernel<1>
              : nv <= 2 ? select_kernel<2>
              : nv <= 4 ? select_kernel<4>
              : nv <= 8 ? select_kernel<8>
                        : select_kernel<16>;
  // tokens beyond the grid are taken by its loop
  const dim3 grid((unsigned)std::min<int64_t>(((int64_t)p.T + 3) / 4, 1 << 20));
  hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, part, nsplit, bias, balance, logits, p.T, p.E, p.k, r, idx, w);
  return hipGetLastError();
}

}  // namespace moe
