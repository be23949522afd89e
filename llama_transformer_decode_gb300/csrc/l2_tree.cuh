// Trees of at most 64 drafted tokens, as a warp handles them: lane i holds tokens i and i + 32.
#pragma once
#include <cuda_runtime.h>

#include "l2_rows.h"

namespace l2 {

typedef unsigned long long u64;

// A tree's parents, parent of token i at from[i] (nullptr: a chain): -1 where it has none.  ok: each comes before its token.
struct TreeParents {
    int lo, hi;
    bool ok;
};
__device__ __forceinline__ TreeParents tree_parents(const int *from, int n) {
    const int lane = threadIdx.x & 31;
    TreeParents t;
    t.lo = lane < n ? (from ? from[lane] : lane - 1) : -1;
    t.hi = lane + 32 < n ? (from ? from[lane + 32] : lane + 31) : -1;
    const bool fine = t.lo >= -1 && t.lo < lane && t.hi >= -1 && t.hi < lane + 32;
    t.ok = __all_sync(0xffffffffu, fine);
    if (!fine) t.lo = t.hi = -1;  // whatever is done with them stays within the tree
    return t;
}

// Bit j of token i's word: j is i or above it.  Paths of twice the length in each of six rounds: a token's word takes that of the token
// at which its path so far ends, and goes on from where that one's ends.
struct TreeWords {
    u64 lo, hi;
};
__device__ __forceinline__ TreeWords tree_words(const TreeParents &t) {
    const int lane = threadIdx.x & 31;
    TreeWords w = {1ull << lane, 1ull << (lane + 32)};
    int jl = t.lo, jh = t.hi;
#pragma unroll 1
    for (int round = 0; round < 6; ++round) {
        auto at = [&](int j, u64 &word, int &next) {  // what token j has
            const u64 a = __shfl_sync(0xffffffffu, w.lo, j & 31), b = __shfl_sync(0xffffffffu, w.hi, j & 31);
            const int c = __shfl_sync(0xffffffffu, jl, j & 31), d = __shfl_sync(0xffffffffu, jh, j & 31);
            word = j < 0 ? 0 : j < 32 ? a : b;
            next = j < 0 ? -1 : j < 32 ? c : d;
        };
        u64 wl, wh;
        int nl, nh;
        at(jl, wl, nl);
        at(jh, wh, nh);
        w.lo |= wl;
        w.hi |= wh;
        jl = nl;
        jh = nh;
    }
    return w;
}
// Token i's word (i the same or not in all lanes).
__device__ __forceinline__ u64 tree_word(const TreeWords &w, int i) {
    const u64 a = __shfl_sync(0xffffffffu, w.lo, i & 31), b = __shfl_sync(0xffffffffu, w.hi, i & 31);
    return i < 32 ? a : b;
}

}  // namespace l2
