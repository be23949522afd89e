// The kernels of attn_walk_16.cuh for one query row per sequence.
#include "attn_walk_16.cuh"

namespace l2 {

// A box must start at a page row and cover whole groups of 8 lines of the swizzle: pages of 8 rows and more that divide a
// tile or are a multiple of one; a tensor's strides are below 2^40 bytes.
bool attn_pages_tc_supported(const PagesAttn &p) {
    const long long lim = 1ll << 40;
    return p.page_size >= 8 && (p.page_size % tc_keys(false) == 0 || tc_keys(false) % p.page_size == 0) && p.row_stride < lim && p.head_stride < lim &&
           p.page_stride < lim && tensor_map_encoder();
}

int attn_pages_16_shift(int hs) { return hs <= 64 ? 5 : 4; }
static_assert(Shape<64, 1>::KT == 1 << 5 && Shape<128, 1>::KT == 1 << 4, "the plan counts tiles by shifts");

cudaError_t launch_attn_pages_16(const PagesAttn &p, cudaLaunchConfig_t cfg) { return launch_16<false>(p, cfg); }

}  // namespace l2
