// The library's rules on sizes behind a C interface, for the tests: which kernels
// a call takes.  Built by tests/kernel_rules.py with the host compiler.
#include "../combine_router_top_amd/csrc/tile_rules.h"

extern "C" {

void rules_train(int64_t cus, int64_t tk, int E, int n, int d, int f, int64_t* out) {
  const moe::TrainPlan p = moe::train_plan(cus, tk, E, n, d, f);
  out[0] = p.up;
  out[1] = p.down;
}

void rules_backward(int64_t cus, int64_t tk, int E, int n, int d, int f, int input, int wants, int64_t* out) {
  const moe::BackwardPlan p = moe::backward_plan(cus, tk, E, n, d, f, input != 0, wants);
  out[0] = p.gate;
  out[1] = p.input;
  out[2] = p.mode;
  out[3] = p.div;
  out[4] = p.units;
  out[5] = p.apart;
}

void rules_i8(int64_t cus, int gated, int segments, int n, int N, int kt, int64_t mean, int64_t all, int64_t most,
              int64_t* out) {
  const moe::I8Plan p = moe::i8_plan(cus, moe::I8Shape{gated != 0, segments != 0, n, N, kt, mean, all, most});
  out[0] = p.stream;
  out[1] = p.tiles;
  out[2] = p.wide;
  out[3] = p.low;
  out[4] = p.blocks;
  out[5] = p.height;
}

}  // extern "C"
