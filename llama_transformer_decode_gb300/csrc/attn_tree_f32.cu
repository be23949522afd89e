// The kernels of attn_walk_f32.cuh for trees of drafted tokens.
#include "attn_walk_f32.cuh"

namespace l2 {

cudaError_t launch_attn_tree_f32(const PagesAttn &p, cudaLaunchConfig_t cfg) { return launch_f32<true>(p, cfg); }

}  // namespace l2
