// How the blocks of a paged attention call divide into its two roles.  Plain C++, so that a test on the CPU runs the same code
// as the plan.
#pragma once
#ifdef __CUDACC__
#define L2_SPLIT_FN __host__ __device__ __forceinline__
#else
#define L2_SPLIT_FN inline
#endif

namespace l2 {

struct RoleSplit {
    int n_tc;    // blocks of the tensor-core role, the first ones
    int per_tc;  // cost a block of it takes
    int per;     // cost a walking warp takes
};

// walk, tc: cost of all tiles of either role.  Blocks go to the roles by cost, at least one to each that has work; a range of either
// is at least least_walk or least_tc.
L2_SPLIT_FN RoleSplit split_roles(int walk, int tc, int blocks, int walk_warps, int least_walk, int least_tc) {
    auto up = [](int a, int b) { return (int)((unsigned)(a + b - 1) / (unsigned)b); };  // a >= 0, b > 0
    RoleSplit r = {0, 1, least_walk};
    if (tc) {
        // n or n + 1 blocks, whichever leaves the slower role less
        const float t = (float)tc, w = (float)walk;
        const int most = blocks - (walk ? 1 : 0);
        int n = (int)((float)blocks * (t / (t + w)));
        n = n < 1 ? 1 : n > most ? most : n;
        auto slower = [&](int k) {
            const float a = t / (float)k, b = walk ? w / (float)(blocks - k) : 0.f;
            return a > b ? a : b;
        };
        if (n < most && slower(n + 1) < slower(n)) ++n;
        const int per = up(tc, n);
        r.per_tc = per > least_tc ? per : least_tc;
        r.n_tc = up(tc, r.per_tc);
    }
    if (walk) {  // without it every block may have gone to the other role
        const int per = up(walk, (blocks - r.n_tc) * walk_warps);
        if (per > r.per) r.per = per;
    }
    return r;
}

}  // namespace l2
