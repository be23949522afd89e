// The kernels of attn_walk_16.cuh for trees of drafted tokens.
#include "attn_walk_16.cuh"

namespace l2 {

int attn_tree_16_shift(int hs, int team) { return hs <= 64 || team > 1 ? 5 : 4; }
static_assert(Shape<64, 1>::KT == 1 << 5 && Shape<128, 1>::KT == 1 << 4 && Shape<64, 2>::KT == 1 << 5 && Shape<128, 4>::KT == 1 << 5,
              "the plan counts tiles by shifts");

cudaError_t launch_attn_tree_16(const PagesAttn &p, cudaLaunchConfig_t cfg) { return launch_16<true>(p, cfg); }

}  // namespace l2
