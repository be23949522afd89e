// The plan of a paged attention call: lengths of the sources and the numbering of their tiles and items.  Built by one
// block of NT threads, either a kernel of its own or, for calls of few sources, every block of the kernel for itself.
#pragma once
#include "../../include/l2.h"
#include "attn_pages.cuh"
#include "attn_split.h"

namespace l2 {

// Least cost of a range, an item's start and two tiles: fewer cost more to write and merge as parts than the parallel reading gains.  (And
// at least the distance of two tiles of any kind, see walker_of.)
__device__ __forceinline__ int tc_min_per(int hs, bool f32) { return kTcItemCost + tc_cost(2 * kTcRows, hs, f32); }
// An item of k tiles goes to sqrt(13 k) warps at most (48 for 180 tiles, 285 for 6250): with P warps they take k / P tiles each and
// the merge P parts, a part a thirteenth of a tile's time, and that many make the sum least.
constexpr float kSpread = 1.0f / 13.0f;
static_assert(2 * kCostUnit >= kMaxTileCost, "every walker between an item's first and last must hold a tile of it");

template <int NT, int MAX>
struct PlanScratch {
    int minlen[MAX], mintc[MAX], gstart[MAX + 1], len[MAX], group[MAX], seq[MAX];
    int2 sums[2][32];
    int spread;
    unsigned long long cost[2];
};

// Places are numbered in 32 bits; a walker's range ends at most as far beyond the last as it is long.
constexpr long long kMostCost = 1ll << 30;

// Exclusive prefix sums of both components over the block, and the totals; buf: one int2 a warp, not used by another scan.
template <int NT>
__device__ __forceinline__ int2 plan_scan(int2 v, int2 *total, int2 *buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto warp_scan = [&](int2 x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
            if (lane >= o) {
                x.x += a;
                x.y += b;
            }
        }
        return x;
    };
    const int2 x = warp_scan(v);
    if (lane == 31) buf[warp] = x;
    __syncthreads();
    const int2 s = warp_scan(lane < NT / 32 ? buf[lane] : make_int2(0, 0));
    total->x = __shfl_sync(0xffffffffu, s.x, 31);
    total->y = __shfl_sync(0xffffffffu, s.y, 31);
    const int bx = __shfl_sync(0xffffffffu, s.x, (warp + 31) & 31), by = __shfl_sync(0xffffffffu, s.y, (warp + 31) & 31);
    return make_int2((warp ? bx : 0) + x.x - v.x, (warp ? by : 0) + x.y - v.y);
}

// MAX: most groups or rows (MAX <= NT).  Ends with a barrier.  report: sets the status word when the call is bad.  WIDE: calls with p.wide
// are among those planned; they have a plan kernel (in the attention kernels the sum would cost every call: 155.7 us against 154.4).
// TREE: groups are sequences with trees of drafted tokens.  A group's keys, but for whole tiles that go to the tensor cores, are one
// source then: which of the last ones a row sees is the walk's matter.
template <int NT, int MAX, bool TREE, bool WIDE = false>
__device__ __forceinline__ void plan_build(const PagesAttn &p, const Plan &pl, PlanScratch<NT, MAX> &sc, bool report) {
    const int i = threadIdx.x, S = TREE ? p.G : p.G + p.B, gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    const bool f32 = p.dtype == L2_F32;
    // pairs and start of an item, tiles of 8 KB that one of its tiles is
    const int pairs = TREE ? kM * p.team : kM, start = TREE ? item_cost(true, p.team) : kItemCost, units = TREE ? p.tile_units : 1;
    bool bad = false;
    int len = 0, seq = 0, P = 0, a0 = 0;
    constexpr int kOwn = TREE ? (kPagesMaxCall + NT - 1) / NT : 1;  // parents that a thread looks at
    int parent[kOwn];
    if constexpr (TREE) {
        int a1 = 0;
        if (i < p.G) {
            seq = p.seqs[i];
            a0 = p.group_starts[i];
            a1 = p.group_starts[i + 1];
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (p.parents && k * NT + i < p.B) parent[k] = p.parents[k * NT + i];
        if (i < p.G) {
            bad = seq < 0 || seq >= p.n_seqs;
            if (!bad) len = p.lens[seq];
            bad |= a0 < 0 || a1 < a0 || a1 > p.B || a1 - a0 > kTreeNodes || (i == 0 && a0 != 0);
            bad |= len < a1 - a0 || len > p.max_pages * p.page_size;
            sc.gstart[i] = a0;
            if (i == p.G - 1) sc.gstart[p.G] = a1;
            sc.len[i] = len;
            sc.seq[i] = seq;
            sc.minlen[i] = len - (a1 - a0);  // committed rows
        }
        if (i == 0) {
            sc.spread = 0;
            sc.cost[0] = sc.cost[1] = 0;
        }
    } else {
        // what depends on nothing is loaded before the lengths, which depend on seqs
        if (i < p.G) P = p.prefix_lens[i];
        if (p.G && i <= p.G) a0 = p.group_starts[i];
        if (i < p.B) {
            seq = p.seqs ? p.seqs[i] : i;
            bad = seq < 0 || seq >= p.n_seqs;
            if (!bad) len = p.lens[seq];
            bad |= len < 0 || len > p.max_pages * p.page_size;
            sc.len[i] = len;
            sc.seq[i] = seq;
        }
        if (i == 0) {
            sc.spread = 0;
            sc.cost[0] = sc.cost[1] = 0;
        }
        if (p.G) {
#pragma unroll 1
            for (int g = i; g <= p.G; g += NT) {
                const int a = g == i ? a0 : p.group_starts[g];
                bad |= (g == 0 && a != 0) || (g == p.G && a != p.B) || a < 0 || a > p.B;
                sc.gstart[g] = a;
            }
            bad |= P < 0;
            __syncthreads();
            if (i < p.G) {
                const int rows = sc.gstart[i + 1] - sc.gstart[i];
                bad |= rows < 0;
                sc.minlen[i] = rows < 2 ? 0 : P;  // a row alone has nothing to share: all its keys are its own
            }
        }
    }
    auto refused = [&]() {
        if (!__syncthreads_or(bad)) return false;
        if (i < kHdrInts) pl.hdr[i] = i == kHdrPer || i == kHdrTcPer ? 1 : 0;
        if (i == 0 && report) atomicOr(p.err, L2_PAGES_ERR_ARGS);
        __syncthreads();
        return true;
    };
    if (refused()) return;
    int2 tc_all = make_int2(0, 0);
    if constexpr (TREE) {
        // every parent comes before its token, in the same tree
        if (p.parents) {
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                const int r = k * NT + i;
                if (r >= sc.gstart[p.G]) continue;
                int lo = 0, hi = p.G;
#pragma unroll 1
                while (hi - lo > 1) {
                    const int m = (lo + hi) >> 1;
                    sc.gstart[m] <= r ? lo = m : hi = m;
                }
                bad |= parent[k] < -1 || parent[k] >= r - sc.gstart[lo];
            }
            if (refused()) return;
        }
    } else if (p.G) {
        if (i < p.B) {
            int lo = 0, hi = p.G;  // the group of the row: the last that starts at or before it
#pragma unroll 1
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                sc.gstart[m] <= i ? lo = m : hi = m;
            }
            atomicMin(&sc.minlen[lo], len);
            sc.group[i] = pl.group[i] = lo;
        }
        __syncthreads();
    }
    if (WIDE && p.wide) {
        // sequences as long as their tables would not do: what these cost, with every prefix in both roles
        auto tiles = [&](int keys) { return (long long)((keys + (1 << p.tile_shift) - 1) >> p.tile_shift); };
        long long walk = 0, tc = 0;
        if (!TREE && i < p.B) walk = cdiv(gq, kM) * (kItemCost + kMaxTileCost * tiles(len - (p.G ? sc.minlen[sc.group[i]] : 0)));
        if (i < p.G) {
            const int n = (sc.gstart[i + 1] - sc.gstart[i]) * gq;
            walk += cdiv(n, pairs) * (start + (TREE ? kMaxTreeTileCost : kMaxTileCost) * tiles(TREE ? sc.len[i] : sc.minlen[i]));
            tc = tc_runs(n, f32) * (kTcItemCost + tc_cost(n, p.head_size, f32) * (long long)(sc.minlen[i] / tc_keys(f32)));
        }
        if (walk) atomicAdd(&sc.cost[0], (unsigned long long)walk * p.n_kv_heads);
        if (tc) atomicAdd(&sc.cost[1], (unsigned long long)tc * p.n_kv_heads);
        __syncthreads();
        bad = max(sc.cost[0], sc.cost[1]) > (unsigned long long)kMostCost;
        if (refused()) return;
    }
    if (p.G) {
        // prefixes worth it go to the tensor cores in whole tiles; what is left of them stays with the warps
        const int n = i < p.G ? (sc.gstart[i + 1] - sc.gstart[i]) * gq : 0;
        int full = i < p.G && p.tc ? sc.minlen[i] / tc_keys(f32) : 0;
        int2 before = make_int2(0, 0);
        if (p.tc) {
            if (!tc_worth(p, n, full * tc_keys(f32))) full = 0;
            if (full)
                before = make_int2((kTcItemCost + full * tc_cost(n, p.head_size, f32)) * tc_runs(n, f32) * p.n_kv_heads,
                                   tc_head_rows(n, f32) * p.n_kv_heads);
            before = plan_scan<NT>(before, &tc_all, sc.sums[0]);
        }
        if (i < p.G) {
            pl.tc_t0[i] = before.x;
            pl.tc_kt[i] = full;
            pl.tc_r0[i] = before.y;
            sc.mintc[i] = full * tc_keys(f32);
        }
        __syncthreads();
    }
    int2 all = make_int2(0, 0);
#pragma unroll 1
    for (int s0 = 0; s0 < S; s0 += NT) {
        const int s = s0 + i;
        Source e = {};
        if (s < p.G) {
            e.key0 = sc.mintc[s];
            e.key1 = TREE ? sc.len[s] : sc.minlen[s];
            e.row0 = sc.gstart[s];
            e.rows = sc.gstart[s + 1] - e.row0;
            if (TREE) {
                e.seq = sc.seq[s];
                if (!e.rows) e.key1 = e.key0;
            }
        } else if (s < S) {
            e.row0 = s - p.G;
            e.rows = 1;
            e.key0 = p.G ? sc.minlen[sc.group[e.row0]] : 0;
            e.key1 = sc.len[e.row0];
        }
        if (!TREE && e.rows > 0) e.seq = sc.seq[e.row0];
        e.kt = (e.key1 - e.key0 + (1 << p.tile_shift) - 1) >> p.tile_shift;
        e.cost = TREE ? tree_tile_cost(p.dtype, min(e.rows * gq, kM), p.team, units) : tile_cost(p.dtype, min(e.rows * gq, kM));
        const int items = e.kt ? (e.rows * gq + pairs - 1) / pairs * p.n_kv_heads : 0;
        if (items) atomicMax(&sc.spread, (int)((float)e.cost * sqrtf((float)e.kt * kSpread)));
        int2 here;
        const int2 before = plan_scan<NT>(make_int2(items * (start + e.kt * e.cost), items), &here, sc.sums[1]);
        e.t0 = all.x + before.x;
        e.i0 = all.y + before.y;
        if (s < S) pl.src[s] = e;
        all.x += here.x;
        all.y += here.y;
        if (s0 + NT < S) __syncthreads();
    }
    if (i == 0) {
        const int cost = all.x, tc = tc_all.x;
        const int least = TREE ? max(2 * kCostUnit * units, tree_tile_cost(p.dtype, kM, p.team, units)) : 2 * kCostUnit;
        const RoleSplit r = split_roles(cost, tc, p.num_sms, TREE ? walk_warps(f32, p.team) / p.team : kWalkWarps, max(start + least, sc.spread),
                                        tc_min_per(p.head_size, f32));
        pl.src[S].t0 = cost;
        pl.hdr[kHdrCost] = cost;
        pl.hdr[kHdrPer] = r.per;
        pl.hdr[kHdrTcCost] = tc;
        pl.hdr[kHdrTcPer] = r.per_tc;
        pl.hdr[kHdrTcBlocks] = r.n_tc;
        if (p.G) pl.tc_t0[p.G] = tc;
        pl.hdr[kHdrOk] = 1;
    }
    __syncthreads();
}

// What the merge needs of each row, from a plan that is complete.
template <int NT, bool TREE>
__device__ __forceinline__ void plan_rows(const PagesAttn &p, const Plan &pl, RowPlan *rows) {
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += NT) {
        RowPlan r = {};
        if constexpr (!TREE) {
            const Source &o = pl.src[p.G + b];
            r.own_t0 = o.t0;
            r.own_i0 = o.i0;
            r.own_kt = o.kt;
            r.own_cost = o.cost;
        }
        if (p.G && pl.hdr[kHdrOk]) {
            int g = 0;
            if constexpr (TREE) {
                int hi = p.G;  // the last group that starts at or before the row
#pragma unroll 1
                while (hi - g > 1) {
                    const int m = (g + hi) >> 1;
                    pl.src[m].row0 <= b ? g = m : hi = m;
                }
                r.behind = b >= pl.src[g].row0 + pl.src[g].rows;
            } else {
                g = pl.group[b];
            }
            const Source &e = pl.src[g];
            r.rest_t0 = e.t0;
            r.rest_i0 = e.i0;
            r.rest_kt = e.kt;
            r.rest_cost = e.cost;
            r.tc_t0 = pl.tc_t0[g];
            r.tc_kt = pl.tc_kt[g];
            r.tc_r0 = pl.tc_r0[g];
            r.group_rows = e.rows;
            r.row_in_group = b - e.row0;
        }
        rows[b] = r;
    }
}

// The plan as a kernel's block uses it: built here (mem: kPlanSmem bytes, scratch: free until the caller's first
// use of it; `keep`: also left in the workspace for the merge), or the workspace's.
template <int NT, bool TREE>
__device__ __forceinline__ Plan plan_here(const PagesAttn &p, void *mem, void *scratch, bool keep) {
    if (!p.plan_in_block) return plan_of(p.plan, p.B, p.G);
    const Plan pl = plan_of(mem, TREE ? 0 : p.B, p.G);  // a tree's rows have no sources of their own
    plan_build<NT, kPlanInBlock, TREE>(p, pl, *static_cast<PlanScratch<NT, kPlanInBlock> *>(scratch), keep);
    if (keep) {
        const Plan out = plan_of(p.plan, p.B, p.G);
        if (threadIdx.x < kHdrInts) out.hdr[threadIdx.x] = pl.hdr[threadIdx.x];
        plan_rows<NT, TREE>(p, pl, out.row);
    }
    return pl;
}

}  // namespace l2
