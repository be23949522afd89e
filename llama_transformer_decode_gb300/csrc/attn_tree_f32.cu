// The kernels of attn_walk_f32.cuh for trees of drafted tokens.
#include "attn_walk_f32.cuh"

namespace l2 {

int attn_tree_f32_shift(int hs, int team) { return hs <= 32 ? 5 : (hs <= 64 ? 4 : 3) + (team > 1 ? 1 : 0); }
static_assert(ShapeF<32, 4>::KT == 1 << 5 && ShapeF<64, 1>::KT == 1 << 4 && ShapeF<64, 2>::KT == 1 << 5 && ShapeF<128, 1>::KT == 1 << 3 &&
              ShapeF<128, 4>::KT == 1 << 4, "the plan counts tiles by shifts");

cudaError_t launch_attn_tree_f32(const PagesAttn &p, cudaLaunchConfig_t cfg) { return launch_f32<true>(p, cfg); }

}  // namespace l2
