// The rules of the 4-bit products behind a C interface, for the tests.  Built by
// tests/rules_4bit.py with the host compiler.
#include "../combine_router_top_amd/csrc/tile_rules.h"

extern "C" void rules_w4(int64_t cus, int gated, int segments, int n, int N, int kb, int64_t mean, int64_t all, int64_t most,
                         int64_t* out) {
  const moe::W4Plan p = moe::w4_plan(cus, moe::W4Shape{gated != 0, segments != 0, n, N, kb, mean, all, most});
  out[0] = p.tiles;
  out[1] = p.bm;
  out[2] = p.parts;
  out[3] = p.per;
  out[4] = p.wide;
  out[5] = p.low;
  out[6] = p.blocks;
  out[7] = p.waves;
  out[8] = p.ahead;
}
