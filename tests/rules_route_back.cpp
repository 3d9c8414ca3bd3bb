// The rules of the router's gradients behind a C interface, for tests/test_route_back_choice.py,
// which builds it with the host compiler.
#include "../combine_router_top_amd/csrc/tile_rules.h"

extern "C" int rules_route_few(int64_t cus, int64_t T, int d) { return moe::route_few(cus, T, d); }
extern "C" int rules_route_shares(int64_t cus, int64_t T, int d, int E) { return moe::route_shares(cus, T, d, E); }
