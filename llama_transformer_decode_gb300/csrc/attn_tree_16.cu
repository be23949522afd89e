// The kernels of attn_walk_16.cuh for trees of drafted tokens.
#include "attn_walk_16.cuh"

namespace l2 {

cudaError_t launch_attn_tree_16(const PagesAttn &p, cudaLaunchConfig_t cfg) { return launch_16<true>(p, cfg); }

}  // namespace l2
