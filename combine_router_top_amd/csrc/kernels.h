// Internal launchers of libmoe (host functions defined next to their kernels).
// All take a validated problem and launch asynchronously on `st`.
#pragma once

#include <hip/hip_runtime.h>

#include "common.h"

namespace moe {

// route.hip
size_t route_ws_bytes(const Prob& p);
// chunk_hist (or NULL): the dispatch chunk histograms (hist_elems int32 =
// ceil(T k / 1024) * E).  Where the router kernel supports it, it clears them
// and top-k counts its selections into them; *hist_done (if given) says
// whether that happened, so that dispatch can skip its histogram kernel.
hipError_t launch_route(const Prob& p, const void* x, const void* wg, const float* bias,
                        float* logits, int32_t* idx, float* w, void* ws, hipStream_t st,
                        int32_t* chunk_hist = nullptr, int64_t hist_elems = 0,
                        bool* hist_done = nullptr);

// The router's product alone: fp32 sums [splits][T][E] into ws (route_ws_bytes).
int route_splits(const Prob& p);
hipError_t launch_route_product(const Prob& p, const void* x, const void* wg, void* ws, hipStream_t st);

// select.hip: how experts are chosen from their logits.
struct SelectRule {
  int softmax;       // scores: softmax, else sigmoid
  int groups, topk_groups, group_top;
  int renorm;
  int by_logit;      // softmax without a bias: the logits order the experts
  int lanes;         // lanes that work on a group: 64 / groups, down to a power of two
  float scale;
};
// part: fp32 sums [nsplit][T][E]; logits (or NULL) receives their total plus bias.
hipError_t launch_select(const Prob& p, const SelectRule& r, const float* part, int nsplit, const float* bias,
                         const float* balance, float* logits, int32_t* idx, float* w, hipStream_t st);

// route_backward.hip: gradients of the router; any output may be NULL.
size_t route_backward_ws_bytes(const Prob& p);
hipError_t launch_route_backward(const Prob& p, const SelectRule& r, const void* x, const void* wg, const float* logits,
                                 const int32_t* idx, const float* dw, const void* dx_add, float* dlogits, void* dx,
                                 void* dwg, float* dbias, void* ws, hipStream_t st);

// dispatch.hip
size_t dispatch_ws_bytes(const Prob& p);
// hist_ready: ws already holds the chunk histograms (filled by top-k), so the
// histogram kernel is skipped.
// w_in / rscale (both or neither): rscale[inv[a]] = w_in[a] for every local
// assignment a (the routing weight of each packed row).
hipError_t launch_dispatch_index(const Prob& p, const int32_t* idx, int32_t* counts_all,
                                 int32_t* offsets, int32_t* perm, int32_t* inv, void* ws,
                                 hipStream_t st, bool hist_ready = false,
                                 const float* w_in = nullptr, float* rscale = nullptr);
// Zero counts_all [E] and offsets [n+1] (either may be NULL): the index of an
// empty batch.  launch_dispatch_index does this itself when T = 0.
hipError_t launch_clear_index(const Prob& p, int32_t* counts_all, int32_t* offsets, hipStream_t st);
// Static per-device scratch of the allocation-free dispatch: its size, and its
// device address on the current device (looked up once per device).
size_t dispatch_scratch_bytes();
hipError_t dispatch_scratch(void** out);
// Gather rows of the local experts [e_begin, e_end) (0-based local indices).
hipError_t launch_gather(const Prob& p, const void* x, const int32_t* offsets,
                         const int32_t* perm, void* x_packed, int e_begin, int e_end,
                         hipStream_t st);

// Padded fixed-capacity layout: n * capacity rows (see dispatch.hip); the
// workspace holds the unpadded index plus the dispatch workspace.
size_t dispatch_padded_ws_bytes(const Prob& p);
hipError_t launch_dispatch_padded(const Prob& p, int capacity, const int32_t* idx,
                                  int32_t* counts_all, int32_t* offsets, int32_t* perm,
                                  int32_t* inv, const void* x, void* x_packed, void* ws,
                                  hipStream_t st);

// expert_gemm.hip: GEMMs over the segments of local experts [e_begin, e_end).
// With perm (bf16 only, T * d * 2 < 2^32), x_packed is x itself and GEMM-1
// gathers its rows through perm (packed row p = token perm[p] / k).
size_t expert_gemm_ws_bytes(const Prob& p);
// With rscale (packed-row weights), y_packed row p is rnd(rscale[p] * (h W2)).
hipError_t launch_expert_gemm(const Prob& p, const void* x_packed, const int32_t* offsets,
                              const void* w1, const void* w3, const void* w2, void* h,
                              void* y_packed, void* ws, int e_begin, int e_end, hipStream_t st,
                              const int32_t* perm = nullptr, const float* rscale = nullptr);

// expert_train.hip: the training forward pass.
hipError_t launch_expert_gemm_train(const Prob& p, const void* x_packed, const int32_t* offsets,
                                    const void* w1, const void* w3, const void* w2, void* g, void* u,
                                    void* h, void* y_packed, hipStream_t st);

// expert_gemm.hip: GEMM C = rnd(A B) with a release flag per 256 x 256 tile
int64_t gemm_signal_tiles(int M, int N);
hipError_t launch_gemm_signal(int M, int N, int K, const void* A, const void* B, void* C,
                              uint32_t* flags, uint32_t epoch, int system_scope, hipStream_t st);
// tile_forward.hip: copy each tile of C to dst once its flag reads epoch
hipError_t launch_tile_forward(int M, int N, const void* C, void* dst, const uint32_t* flags,
                               uint32_t epoch, uint32_t spin_limit, int system_scope,
                               uint32_t* timeouts, int workgroups, hipStream_t st);

// combine.hip
hipError_t launch_combine(const Prob& p, const void* y_packed, const int32_t* inv,
                          const float* w, void* y, hipStream_t st);

// Backward pass of combine; w NULL: unit weights, dw NULL: not wanted (then
// y_packed is not read).
hipError_t launch_combine_backward(const Prob& p, const void* dy, const void* y_packed, const int32_t* inv,
                                   const float* w, void* dy_packed, float* dw, hipStream_t st);

// Compute units of the device (the first one asked about: one process drives one
// kind), and the grid of a persistent kernel over
// `tiles` tiles: a multiple of 8 (one share per XCD) of at most that many.
int device_cus();
inline unsigned st_grid(int64_t tiles) {
  const int64_t most = device_cus() >= 8 ? device_cus() / 8 * 8 : 8;
  const int64_t want = (tiles + 7) / 8 * 8;
  return (unsigned)(want < most ? (want < 8 ? 8 : want) : most);
}

// expert_backward.hip: gradients of the expert FFNs (any output may be NULL).
// T = 0 writes zeros to the wanted weight gradients.
size_t expert_backward_ws_bytes(const Prob& p);
hipError_t launch_expert_backward(const Prob& p, const void* x, const int32_t* offsets, const void* w1,
                                  const void* w3, const void* w2, const void* g, const void* u, const void* h,
                                  const void* dy, void* dx, void* dw1, void* dw3, void* dw2, void* ws, hipStream_t st);

// expert_i8.hip: 8-bit products.  Rows of x (dtype 0 fp32, 1 bf16) to int8 rows
// of ldq bytes and a scale each; limit (or NULL): device row count.
hipError_t launch_quantize_rows(const void* x, int dtype, int64_t rows, int K, int64_t ldq, void* q, float* s,
                                const int32_t* limit, hipStream_t st);
size_t packed_i8_bytes(int n, int K, int N);
hipError_t launch_pack_i8(int n, int K, int N, const void* w, void* packed, hipStream_t st);
hipError_t launch_quantize_weights(int n, int K, int N, int dtype, const void* w, void* packed, float* s,
                                   hipStream_t st);
hipError_t launch_gemm_i8(int M, int N, int K, const void* a, const float* sa, const void* packed, const float* sb,
                          void* c, int out_dtype, hipStream_t st);
size_t expert_i8_ws_bytes(const Prob& p);
hipError_t launch_expert_i8(const Prob& p, const void* x, const int32_t* offsets, const void* q1, const float* s1,
                            const void* q3, const float* s3, const void* q2, const float* s2, void* h, void* y,
                            void* ws, hipStream_t st);

// expert_4bit.hip: products with 4-bit weights in groups of `group` along K; zero
// points may be NULL (8).
size_t packed_4bit_bytes(int n, int K, int N);
hipError_t launch_pack_4bit(int n, int K, int N, const void* w, void* packed, hipStream_t st);
hipError_t launch_quantize_4bit(int n, int K, int N, int group, int dtype, const void* w, void* packed, void* scale,
                                void* zero, hipStream_t st);
size_t gemm_4bit_ws_bytes(int M, int N, int K);
hipError_t launch_gemm_4bit(int M, int N, int K, int group, const void* a, const void* packed, const void* scale,
                            const void* zero, void* c, int out_dtype, void* ws, hipStream_t st);
struct Weights4 {
  const void* w;      // packed [n]
  const void* scale;  // bf16 [n][groups][N]
  const void* zero;   // uint8 [n][groups][N] or NULL
};
size_t expert_4bit_ws_bytes(const Prob& p);
hipError_t launch_expert_4bit(const Prob& p, int group, const void* x, const int32_t* offsets, const Weights4& w1,
                              const Weights4& w3, const Weights4& w2, void* h, void* y, void* ws, hipStream_t st);

}  // namespace moe
