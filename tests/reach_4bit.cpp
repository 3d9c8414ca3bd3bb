// Scalar offsets of the 4-bit products' loads behind a C interface, for tests/test_4bit_reach.py,
// which builds it with the host compiler.
#include "../combine_router_top_amd/csrc/tile_rules.h"

extern "C" uint32_t reach_offset(uint32_t off, uint32_t size) { return moe::st_offset(off, size); }
extern "C" int reach_block(int i, int n) { return moe::st_upto(i, n); }
