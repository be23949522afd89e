// Reads "walk tc blocks warps least_walk least_tc" lines, prints "n_tc per_tc per": csrc/attn_split.h as the plan runs it.
#include <cstdio>

#include "attn_split.h"

int main() {
    int walk, tc, blocks, warps, least_walk, least_tc;
    while (scanf("%d %d %d %d %d %d", &walk, &tc, &blocks, &warps, &least_walk, &least_tc) == 6) {
        const l2::RoleSplit r = l2::split_roles(walk, tc, blocks, warps, least_walk, least_tc);
        printf("%d %d %d\n", r.n_tc, r.per_tc, r.per);
    }
    return 0;
}
