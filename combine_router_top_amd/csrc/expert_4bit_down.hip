// Plain 4-bit products on tiles: C = rnd(A W).
#include "w4_tile.h"

namespace moe {

hipError_t launch_4bit_tiles_down(const W4Args& p, int group, int bm, int64_t rows_max, bool f32out, hipStream_t st) {
  return f32out ? launch_w4_tiles<false, true>(p, group, bm, rows_max, st)
                : launch_w4_tiles<false, false>(p, group, bm, rows_max, st);
}

}  // namespace moe
