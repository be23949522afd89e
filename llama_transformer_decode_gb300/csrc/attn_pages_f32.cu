// The kernels of attn_walk_f32.cuh for one query row per sequence.
#include "attn_walk_f32.cuh"

namespace l2 {

int attn_pages_f32_shift(int hs) { return hs <= 32 ? 5 : hs <= 64 ? 4 : 3; }
static_assert(ShapeF<32, 1>::KT == 1 << 5 && ShapeF<64, 1>::KT == 1 << 4 && ShapeF<128, 1>::KT == 1 << 3, "the plan counts tiles by shifts");

cudaError_t launch_attn_pages_f32(const PagesAttn &p, cudaLaunchConfig_t cfg) { return launch_f32<false>(p, cfg); }

}  // namespace l2
