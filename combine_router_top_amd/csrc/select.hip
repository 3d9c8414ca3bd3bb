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
#include "wave_reduce.h"

namespace moe {

// The choice is made in fp32, with every comparison that decides it watched: where two
// values that matter are nearer to each other than twice their error (2^-21 of 1 + |c|
// for sigmoid scores, 2^-19 for softmax scores, whose sum has up to 22 roundings), it is
// made again in fp64: among the candidates that are that near (sigmoid scores), or from
// the start (near groups, softmax scores with a bias).  That happens to about one token
// in 500 with 256 experts, without groups or in 8.  Groups that are not whole lanes, a power of
// two up to 16 of them, have no fp32 form: every token goes through fp64 (4096 tokens of 160
// experts in 8 groups 14.5 us, of 384 in 8 25.7, of 256 in 2 14.4, against 10.9 of 256 in 8).
// Comparisons of logits are exact.
constexpr double SEL_LOW = -1e300;        // experts that come last, in fp64
constexpr float SEL_LOW_F = -3.402823466e38f;   // in fp32 sums of groups; single experts that come last have -inf

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

__device__ __forceinline__ uint32_t reduce_max(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ float reduce_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float reduce_sum(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}

// A value that is no number, or below, is the lowest.
__device__ __forceinline__ double sel_floor(double c) { return c >= SEL_LOW ? c : SEL_LOW; }

// The two largest values a >= b of two pairs.
template <class T>
struct Top2 {
  T a, b;
};
template <class T>
__device__ __forceinline__ Top2<T> merge(const Top2<T>& p, const Top2<T>& q) {
  return Top2<T>{max(p.a, q.a), max(min(p.a, q.a), max(p.b, q.b))};
}

// Groups that stay, as a mask with bit g L of each (L = r.lanes): the groups with fewer than
// topk_groups better ones, or as good and before them; `mine` is the value of the group of
// lanes g L .. g L + L - 1.  In fp32, that value may be off by `error`, in proportion to the sizes
// of its members (they may cancel), and `close` is set where that could change what stays;
// `masked`: a member comes last, and the value may be any lower.
template <class T>
__device__ __forceinline__ uint64_t open_groups(T mine, const SelectRule& r, float error, bool masked, bool& close) {
  const int g = (threadIdx.x & 63) / r.lanes;
  int better = 0;
  for (int q = 0; q < r.groups; ++q) {
    T v;
    if constexpr (sizeof(T) == 4) v = lane_of(mine, q * r.lanes);
    else v = __shfl(mine, q * r.lanes);
    better += v > mine || (v == mine && q < g);
  }
  const bool in = g < r.groups, stay = in && better < r.topk_groups;
  if constexpr (sizeof(T) == 4)
    if (r.topk_groups < r.groups) {   // the least that one that stays can be, the most that another can
      const float worst = -reduce_max(!stay ? -INFINITY : masked ? INFINITY : error - mine);
      const float best = reduce_max(in && !stay ? mine + error : -INFINITY);
      close |= !(worst > best);
    }
  return __ballot(stay);
}

// Sums of the K splits, the logits' bias; expert NV l + j of lane l, -inf past the last.
template <int NV>
__device__ __forceinline__ void token_logits(const float* __restrict__ part, int nsplit,
                                             const float* __restrict__ bias, float* __restrict__ logits_out, int64_t t,
                                             int64_t sstride, int E, float (&l)[NV]) {
  const int e0 = NV * (threadIdx.x & 63);
  const float* pt = part + t * E;
  const bool quads = NV % 4 == 0 && E % 4 == 0 && (reinterpret_cast<uintptr_t>(part) & 15) == 0;
  auto row = [&](const float* p, float (&v)[NV]) {
    if (quads) {
#pragma unroll
      for (int j = 0; j < NV; j += 4) {
        f32x4 q = f32x4{0.f, 0.f, 0.f, 0.f};
        if (e0 + j < E) q = *reinterpret_cast<const f32x4*>(p + e0 + j);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < NV) v[j + i] = q[i];
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = e0 + j < E ? p[e0 + j] : 0.f;
    }
  };
  row(pt, l);
  for (int s = 1; s < nsplit; s += 4) {   // four splits on their way together
    float v[4][NV];
#pragma unroll
    for (int u = 0; u < 4; ++u) row(pt + (int64_t)min(s + u, nsplit - 1) * sstride, v[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < NV; ++j) l[j] = s + u < nsplit ? l[j] + v[u][j] : l[j];
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = e0 + j;
    if (e < E) {
      if (bias) l[j] += bias[e];
      if (logits_out) logits_out[t * E + e] = l[j];
    } else {
      l[j] = -INFINITY;
    }
  }
}

// The k experts of a token in fp64; lane q < k returns its q-th, or 0.
template <int NV>
__device__ __forceinline__ int choose_exact(const float (&l)[NV], const float* __restrict__ balance, int E, int k,
                                         const SelectRule& r, double* value) {
  const int lane = threadIdx.x & 63, e0 = NV * lane;
  float top = l[0];
#pragma unroll
  for (int j = 1; j < NV; ++j) top = fmaxf(top, l[j]);
  top = wave_max_of(top);
  double c[NV], total = 0.0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] = r.softmax ? (e0 + j < E ? exp((double)l[j] - (double)top) : 0.0) : 1.0 / (1.0 + exp(-(double)l[j]));
    total += c[j];
  }
  total = r.softmax ? wave_sum_of(total) : 1.0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] /= total;
    if (balance && e0 + j < E) c[j] += (double)balance[e0 + j];
    c[j] = l[j] == -INFINITY ? SEL_LOW : sel_floor(c[j]);
    if (r.groups > 1 && e0 + j < E) value[e0 + j] = c[j];
    if (r.by_logit) c[j] = sel_floor((double)l[j]);
  }
  lds_wave_order();
  uint64_t open = 0;
  const int per = E / r.groups;
  if (r.groups > 1) {
    const int g = lane / r.lanes;
    Top2<double> v{-INFINITY, -INFINITY};
    if (g < r.groups)
      for (int i = lane % r.lanes; i < per; i += r.lanes) v = merge(v, Top2<double>{value[g * per + i], -INFINITY});
    for (int off = 1; off < r.lanes; off <<= 1) v = merge(v, Top2<double>{__shfl_xor(v.a, off), __shfl_xor(v.b, off)});
    bool close = false;
    open = open_groups<double>(r.group_top == 2 ? v.a + v.b : v.a, r, 0.f, false, close);
  }
  uint64_t key[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = e0 + j;
    key[j] = e < E && (r.groups == 1 || ((open >> (e / per * r.lanes)) & 1)) ? order_key(c[j]) : 0;
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
    const int L = __builtin_ctzll(__ballot(best == m));   // the lowest lane holds the lowest expert
    const int jl = __builtin_amdgcn_readlane(bj, L);
    if (lane == q) mye = NV * L + jl;
    if (lane == L) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j == jl) key[j] = 0;
    }
  }
  lds_wave_order();   // `value` is written again for the next token
  return mye;
}

// One wave per token.  Lane l holds the NV experts NV l .. NV l + NV - 1.  A round of the
// choice is a maximum over the wave, six dependent steps and a way through scalar
// registers; k + 1 rounds, the groups' loop and the weights' two sums follow one another: 256
// experts in 8 groups, 8 of them, one token 6.0 us (without groups 5.4), 4096 tokens 10.9 (9.4).
template <int NV>
__global__ __launch_bounds__(256) void select_kernel(const float* __restrict__ part, int nsplit,
                                                     const float* __restrict__ bias,
                                                     const float* __restrict__ balance,
                                                     float* __restrict__ logits_out, int T, int E, int k, SelectRule r,
                                                     int32_t* __restrict__ idx, float* __restrict__ w) {
  __shared__ double value[4][64 * NV];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e0 = NV * lane;
  const int64_t sstride = (int64_t)T * E;
  const int per = E / r.groups;
  // groups of whole lanes, 2^n up to 16 of them: their two best by DPP
  const bool rows = r.groups > 1 && per % NV == 0 && per / NV <= 16 && ((per / NV) & (per / NV - 1)) == 0 &&
                    per / NV == r.lanes;
  const bool sums = r.softmax && (!r.renorm || !r.by_logit || r.groups > 1);   // scores of all experts are needed
  const float slack = r.softmax ? 0x1p-18f : 0x1p-20f;
  float b[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) b[j] = balance && e0 + j < E ? balance[e0 + j] : 0.f;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < T; t += (int64_t)gridDim.x * 4) {
    float l[NV];
    token_logits<NV>(part, nsplit, bias, logits_out, t, sstride, E, l);
    float top = l[0];
    bool bad = l[0] != l[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) {
      top = fmaxf(top, l[j]);
      bad |= l[j] != l[j];
    }
    float inv = 1.f;   // softmax: 1 over the sum
    if (r.softmax) top = reduce_max(top);
    float c[NV];
    if (sums || !r.softmax) {
      float total = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float z = __builtin_amdgcn_exp2f((r.softmax ? l[j] - top : -l[j]) * 1.4426950408889634f);
        c[j] = r.softmax ? z : __builtin_amdgcn_rcpf(1.0f + z);
        total += c[j];   // experts past the last: exp(-inf) = 0
      }
      if (r.softmax) inv = 1.0f / reduce_sum(total);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (r.softmax) c[j] *= inv;
        c[j] += b[j];
        if (l[j] == -INFINITY || !(c[j] >= SEL_LOW_F)) c[j] = -INFINITY;
      }
    }
    bool close = false;
    uint64_t open = 0;
    if (rows) {
      Top2<float> v{fmaxf(c[0], SEL_LOW_F), SEL_LOW_F};
#pragma unroll
      for (int j = 1; j < NV; ++j) v = merge(v, Top2<float>{c[j], SEL_LOW_F});   // -inf: below both
      if (r.lanes > 1) v = merge(v, Top2<float>{dpp<0xB1>(v.a), dpp<0xB1>(v.b)});
      if (r.lanes > 2) v = merge(v, Top2<float>{dpp<0x4E>(v.a), dpp<0x4E>(v.b)});
      if (r.lanes > 4) v = merge(v, Top2<float>{dpp<0x141>(v.a), dpp<0x141>(v.b)});
      if (r.lanes > 8) v = merge(v, Top2<float>{dpp<0x140>(v.a), dpp<0x140>(v.b)});
      const bool two = r.group_top == 2;
      // each member is off by up to slack / 2 (1 + |c|), their sum by 2^-24 <= slack / 16 of itself more
      const float part = 0.5625f * slack, error = two ? slack + part * fabsf(v.a) + part * fabsf(v.b) : part + part * fabsf(v.a);
      open = open_groups<float>(two ? fmaxf(v.a + v.b, SEL_LOW_F) : v.a, r, error, two && v.b == SEL_LOW_F, close);
    } else if (r.groups > 1) {
      close = true;   // odd groups: in fp64
    }
    uint32_t key[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float v = r.by_logit ? (l[j] == l[j] ? l[j] : -INFINITY) : c[j];
      const bool in = e0 + j < E && (r.groups == 1 || ((open >> (lane & -r.lanes)) & 1));
      key[j] = in ? f32_order_key(v) : 0u;
    }
    int mye = 0;
    float mine = 0.f;   // the logit of lane q's expert, from the lane that holds it
    auto fetch = [&]() {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float v = __shfl(l[j], mye / NV);
        if (mye % NV == j) mine = v;
      }
    };
    bool again = false;   // near candidates
    int count = k;        // candidates
    if (!close) {
      float before = INFINITY;
      for (int q = 0; q < 64; ++q) {
        if (r.by_logit && q == k) break;
        uint32_t bk = key[0];
        int bj = 0;
#pragma unroll
        for (int j = 1; j < NV; ++j)
          if (key[j] > bk) {
            bk = key[j];
            bj = j;
          }
        const uint32_t m = reduce_max(bk);
        if (!r.by_logit) {
          const float v = __uint_as_float((m & 0x80000000u) ? (m & 0x7FFFFFFFu) : ~m);
          // the last ones are alike by definition; m = 0: nothing is left
          const bool near = m != 0 && v != -INFINITY && !(before - v > slack * (1.0f + fabsf(v)));
          if (q >= k && !near) break;
          again |= near;
          before = v;
          count = q + 1;
        }
        const int L = (int)__builtin_ctzll(__ballot(bk == m));
        const int jl = __builtin_amdgcn_readlane(bj, L);
        if (lane == q) mye = NV * L + jl;
        if (lane == L) {
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (j == jl) key[j] = 0;
        }
      }
      close = again && (r.softmax || count == 64);
    }
    if (close) mye = choose_exact<NV>(l, balance, E, k, r, value[wave]);
    fetch();
    if (again && !close) {   // the candidates' order in fp64
      double c64 = -INFINITY;
      if (lane < count) {
        c64 = 1.0 / (1.0 + exp(-(double)mine));
        if (balance) c64 += (double)balance[mye];
        c64 = mine == -INFINITY ? SEL_LOW : sel_floor(c64);
      }
      int rank = lane < count ? 0 : lane;
      for (int q = 0; q < count; ++q) {
        const double v = __shfl(c64, q);
        const int e = __builtin_amdgcn_readlane(mye, q);
        if (lane < count) rank += v > c64 || (v == c64 && e < mye);
      }
      mye = __builtin_amdgcn_ds_permute(4 * rank, mye);
      mine = __int_as_float(__builtin_amdgcn_ds_permute(4 * rank, __float_as_int(mine)));
    }
    float s = 0.f;
    {
      if (r.softmax) {
        // renorm: by the best of the chosen, which a balance may take from far below the row's
        // best, where fp32 holds no scores but their ratios are the weights all the same
        const float from = r.renorm ? reduce_max(lane < k ? mine : -INFINITY) : top;
        s = expf(mine - from);
        if (!r.renorm) s *= inv;
        if (mine == -INFINITY) s = 0.f;   // also where every logit is
      } else {
        // renorm: all by exp(-shift), so that the ratio of tiny scores is theirs
        const float neg = fminf(mine, 0.f);
        float shift = 0.f;
        if (r.renorm) shift = reduce_max(lane < k ? neg : -INFINITY);
        s = expf(neg - shift) / (1.0f + expf(-fabsf(mine)));
        if (mine == -INFINITY) s = 0.f;
      }
    }
    if (r.renorm) {
      const float sum = reduce_sum(lane < k ? s : 0.f);
      s = sum == 0.f ? 0.f : s / sum;
    }
    // softmax of a row with a NaN or a +inf
    if (r.softmax && (__ballot(bad) != 0 || top == INFINITY)) s = NAN;
    if (lane < k) {
      idx[t * k + lane] = mye;
      w[t * k + lane] = s * r.scale;
    }
  }
}

// Up to 128 experts ordered by their logits, without groups, k up to 16: four tokens per
// wave, one in each row of 16 lanes, lane l of a row holding experts NV l .. NV l + NV - 1.
// A round's maximum is four DPP steps for four tokens, against four and a way through
// scalar registers for one: 30011 tokens of 72 experts 25.0 -> 8.3 us.
template <int NV>
__global__ __launch_bounds__(256) void select_rows(const float* __restrict__ part, int nsplit,
                                                   const float* __restrict__ bias, float* __restrict__ logits_out,
                                                   int T, int E, int k, SelectRule r, int32_t* __restrict__ idx,
                                                   float* __restrict__ w) {
  __shared__ f32x2 found[4][4][16];   // expert and logit of a token's q-th choice
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane >> 4, i = lane & 15, e0 = NV * i;
  const int64_t sstride = (int64_t)T * E;
  auto fmax2 = [](float a, float b) { return fmaxf(a, b); };
  auto add = [](float a, float b) { return a + b; };
  auto umax = [](uint32_t a, uint32_t b) { return max(a, b); };
  for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4; t0 < T; t0 += (int64_t)gridDim.x * 16) {
    const int64_t t = t0 + row;
    const bool live = t < T;
    const float* pt = part + (live ? t : T - 1) * E;
    float l[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) l[j] = e0 + j < E ? pt[e0 + j] : 0.f;
    for (int s = 1; s < nsplit; ++s)
#pragma unroll
      for (int j = 0; j < NV; ++j) l[j] += e0 + j < E ? pt[s * sstride + e0 + j] : 0.f;
    bool bad = false;
    float top = -INFINITY;
    uint32_t key[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = e0 + j;
      if (e < E) {
        if (bias) l[j] += bias[e];
        if (logits_out && live) logits_out[t * E + e] = l[j];
      } else {
        l[j] = -INFINITY;
      }
      bad |= l[j] != l[j] || l[j] == INFINITY;
      top = fmaxf(top, l[j]);
      key[j] = e < E ? f32_order_key(l[j] == l[j] ? l[j] : -INFINITY) : 0u;
    }
    top = row_reduce(top, fmax2);
    float total = 1.f;
    if (!r.renorm) {
      total = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) total += __builtin_amdgcn_exp2f((l[j] - top) * 1.4426950408889634f);
      total = row_reduce(total, add);
    }
    for (int q = 0; q < k; ++q) {
      uint32_t bk = key[0];
      int bj = 0;
      float bl = l[0];
#pragma unroll
      for (int j = 1; j < NV; ++j) {
        const bool more = key[j] > bk;
        bk = more ? key[j] : bk;
        bj = more ? j : bj;
        bl = more ? l[j] : bl;
      }
      const uint32_t m = row_reduce(bk, umax);
      const uint32_t holders = (uint32_t)(__ballot(bk == m) >> (16 * row)) & 0xFFFFu;
      if (i == __builtin_ctz(holders)) {   // the lowest lane holds the lowest expert
        found[wave][row][q] = f32x2{__int_as_float(e0 + bj), bl};
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = j == bj ? 0u : key[j];
      }
    }
    const bool any_bad = ((__ballot(bad) >> (16 * row)) & 0xFFFFu) != 0;
    lds_wave_order();
    const f32x2 mine = found[wave][row][i];
    lds_wave_order();   // before the next tokens' choices are written
    float s = i < k && mine[1] != -INFINITY ? expf(mine[1] - top) : 0.f;
    if (r.renorm) total = row_reduce(s, add);
    s = s == 0.f ? 0.f : s / total;
    if (any_bad) s = NAN;
    if (live && i < k) {
      idx[t * k + i] = __float_as_int(mine[0]);
      w[t * k + i] = s * r.scale;
    }
  }
}

hipError_t launch_select(const Prob& p, const SelectRule& r, const float* part, int nsplit, const float* bias,
                         const float* balance, float* logits, int32_t* idx, float* w, hipStream_t st) {
  if (r.by_logit && r.groups == 1 && p.E <= 128 && p.k <= 16) {
    const int nr = (p.E + 15) / 16;
    auto rows = nr <= 1 ? select_rows<1> : nr <= 2 ? select_rows<2> : nr <= 5 ? select_rows<5> : select_rows<8>;
    const dim3 g((unsigned)std::min<int64_t>(((int64_t)p.T + 15) / 16, 8 * (int64_t)device_cus()));
    hipLaunchKernelGGL(rows, g, dim3(256), 0, st, part, nsplit, bias, logits, p.T, p.E, p.k, r, idx, w);
    return hipGetLastError();
  }
  const int nv = (p.E + 63) / 64;
  auto kern = nv <= 1   ? select_kernel<1>
              : nv <= 2 ? select_kernel<2>
              : nv <= 4 ? select_kernel<4>
              : nv <= 8 ? select_kernel<8>
                        : select_kernel<16>;
  // tokens beyond the grid are taken by its loop
  const dim3 grid((unsigned)std::min<int64_t>(((int64_t)p.T + 3) / 4, 8 * (int64_t)device_cus()));
  hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, part, nsplit, bias, balance, logits, p.T, p.E, p.k, r, idx, w);
  return hipGetLastError();
}

}  // namespace moe
