// The gate and up product of the 4-bit experts on tiles: h = rnd(SiLU(x W1) (x W3)).
#include "w4_tile.h"

namespace moe {

hipError_t launch_4bit_tiles_up(const W4Args& p, int group, int bm, int64_t rows_max, hipStream_t st) {
  return launch_w4_tiles<true, false>(p, group, bm, rows_max, st);
}

}  // namespace moe
