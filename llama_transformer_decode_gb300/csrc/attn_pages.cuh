// What the kernels of the paged attention share: the plan, the numbering of the parts they leave for the merge, and
// the copies of a walking warp.
#pragma once
#include <cstddef>
#include <cuda_runtime.h>

#include "l2_device.cuh"
#include "l2_pages.h"
#include "l2_tree.cuh"

namespace l2 {

constexpr int kM = 16;        // (row, head) pairs of a warp's item
constexpr int kTcRows = 128;  // pairs of a tensor-core slot
// Keys of a tensor-core tile and most pairs of an item: 16-bit caches have two slots, fp32 caches one.
__host__ __device__ constexpr int tc_keys(bool f32) { return f32 ? 64 : 128; }
__host__ __device__ constexpr int tc_run(bool f32) { return f32 ? kTcRows : 2 * kTcRows; }

// A walker takes the tiles whose place in the numbering of costs falls into its range.  An item of kt tiles is
// first + kt * cost long: `first` is what starting an item costs.  Tile 0 stands at its beginning, tile k at first + k * cost.
__host__ __device__ __forceinline__ int tile_place(int k, int first, int cost) { return k ? first + k * cost : 0; }

// Plan: a header; the sources of the warps (the groups' prefixes, then the rows' own keys: S = G + B, and an end);
// per group, for the tensor-core role, the cost before it, tiles per item and first row of its parts; the group of
// each row; and, for the merge, what it needs of a row's three sources.
enum { kHdrCost = 0, kHdrPer = 1, kHdrOk = 2, kHdrTcCost = 3, kHdrTcPer = 4, kHdrTcBlocks = 5, kHdrInts = 16 };
struct alignas(16) Source {
    int t0, i0, kt, cost;          // cost and items of the sources before it, tiles per item, cost of a tile
    int key0, key1, row0, rows;    // keys, rows
    int seq, pad[3];               // sequence whose table finds the keys
};
struct alignas(16) RowPlan {
    int own_t0, own_i0, own_kt, own_cost;          // its own keys
    int rest_t0, rest_i0, rest_kt, rest_cost;      // what is left of its group's prefix
    int tc_t0, tc_kt, tc_r0, group_rows;           // the prefix's whole tiles
    int row_in_group, behind, pad[2];              // behind: the last tree, a row that is left as it was
};
struct Plan {
    int *hdr;
    Source *src;
    int *tc_t0, *tc_kt, *tc_r0, *group;
    RowPlan *row;  // in the workspace only
};
__host__ __device__ constexpr size_t plan_bytes(int B, int G) {
    return (kHdrInts * 4 + (size_t)(G + B + 1) * sizeof(Source) + (3 * (size_t)G + 1 + B) * 4 + 127) / 128 * 128;
}
__host__ __device__ inline Plan plan_of(void *base, int B, int G) {
    Plan p;
    p.hdr = static_cast<int *>(base);
    p.src = reinterpret_cast<Source *>(p.hdr + kHdrInts);
    p.tc_t0 = reinterpret_cast<int *>(p.src + G + B + 1);
    p.tc_kt = p.tc_t0 + G + 1;
    p.tc_r0 = p.tc_kt + G;
    p.group = p.tc_r0 + G;
    p.row = reinterpret_cast<RowPlan *>(static_cast<char *>(base) + plan_bytes(B, G));
    return p;
}
// A call of at most this many sources is planned by every block of its kernel for itself, in shared memory: about
// 2 us of latency where a kernel of its own before it costs 6.  Larger calls have such a kernel.
constexpr int kPlanInBlock = 192;
constexpr size_t kPlanSmem = plan_bytes(kPlanInBlock / 2, kPlanInBlock / 2);  // the most for G + B sources, G <= B
constexpr int kTreePlanInBlock = 128;  // sequences with trees, whose rows are no sources
static_assert(plan_bytes(0, kTreePlanInBlock) <= kPlanSmem && kTreePlanInBlock <= kPlanInBlock, "the plan's room");

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (int)((unsigned)(a + b - 1) / (unsigned)b); }  // a >= 0, b > 0

// Most query heads of a KV head; head j of KV head g is first_head(g) + j.
__host__ __device__ __forceinline__ int heads_per_kv(int H, int KV) { return cdiv(H, KV); }
__device__ __forceinline__ int first_head(int g, int H, int KV) { return cdiv(g * H, KV); }

// A total cost T is cut into ranges of `per`: a cost x falls to walker x / per.  per is at least the distance of two tiles, so
// every walker between those of an item's first and last tile holds one of its tiles.
__device__ __forceinline__ int walker_of(int x, int per) { return (int)((unsigned)x / (unsigned)per); }

// Tensor-core items of a group: n pairs (row, head) of one KV head in runs of up to tc_run.  In 16-bit caches a run of up
// to 128 pairs is served by both slots, which take alternate tiles and leave a part of n rows each; of a
// longer one slot 0 takes the first 128.  Parts of walker w and a run: rows
// tc_r0 + (rows of the group's runs before) + tc_run * w of the parts' arrays, which keeps
// them apart: from walker to walker by tc_run rows, from run to run by the run's own.
__host__ __device__ __forceinline__ int tc_runs(int n, bool f32) { return cdiv(n, tc_run(f32)); }
__host__ __device__ __forceinline__ int tc_head_rows(int n, bool f32) {  // of all runs of one KV head
    if (f32) return n;
    const int full = tc_runs(n, false) - 1, last = n - tc_run(false) * full;
    return tc_run(false) * full + (last > kTcRows ? last : 2 * last);
}

// Cost of a tile of an item of n pairs, in quarters of reading it.  16-bit: reading bounds every size.  fp32: the FMAs cost
// what reading does from 5 pairs on, the split products of more than 8 pairs nearly twice that; measured on GB300,
// 1 GB of suffixes of head size 128 / 64: 168 / 167 us at 1 pair, 174 / 167 at 4, 210 / 220 at 8, 318 / 282 at 16.
// Starting an item (its queries, its part) takes a warp 1.25 us where a tile takes 1.55.
constexpr int kCostUnit = 4, kItemCost = 3, kMaxTileCost = 7;
// A tree's item takes longer to start (3 us: its tokens' words, too), and a team of warps is one walker: that many are idle meanwhile.
constexpr int kTreeItemCost = 7;
__host__ __device__ constexpr int item_cost(bool tree, int team) { return (tree ? kTreeItemCost : kItemCost) * team; }
__host__ __device__ __forceinline__ int tile_cost(int dtype, int n) { return dtype != 0 || n <= 4 ? 4 : n <= 8 ? 5 : kMaxTileCost; }
// The same for teams, whose tiles (of `units` 8 KB) keep their warps longer than HBM would take.  32 sequences of 8000 keys in bf16, 8 KV heads of
// 128, 16 / 32 / 64 pairs with 1 / 2 / 4 warps 173 / 217 / 388 us, of 64: 136 with 2, and 4 of 64 132 with 4; fp32, 8 of 3000 and 32 heads of
// 128: 246 / 369 / 720.
__host__ __device__ __forceinline__ int tree_tile_cost(int dtype, int n, int team, int units) {
    if (team == 1) return tile_cost(dtype, n);
    if (dtype == 0) return (team == 2 ? 21 : 41) * units / 2;
    return units == 2 ? (team == 2 ? 10 : 18) : team == 2 ? 7 : 13;
}
constexpr int kMaxTreeTileCost = 41;
// Cost of a tensor-core tile for n pairs of a KV head, in the same unit (a quarter of reading 8 KB, 0.049 us an SM).  A 16-bit tile
// alone, prefix 131072: head size 64, 1.0 to 1.4 us up to 128 pairs, 2.0 to 2.4 above; head size 128, 1.65 (reading) to 1.9, and 2.7
// to 3.3.  Beside walkers, which take HBM, it is longer; over eleven calls with both, prefixes of 4096 to 16384, these costs
// were best or within 3 % of it (64 rows of 32 KV heads: 108 us, 115 with costs a third lower).  fp32, whatever the pairs, 2.4 and
// 3.4, and 4.4 for the planning, for the same reason (32 KV heads of 32 pairs, prefix 2048: 189 us with 3.0, 161 with 3.7, 153
// with 4.4 or more).  Starting an item: its queries, its part, and the pipeline's filling.
constexpr int kTcItemCost = 80;
__host__ __device__ __forceinline__ int tc_cost(int n, int hs, bool f32) {
    if (f32) return hs > 64 ? 90 : 50;
    return n > kTcRows ? (hs > 64 ? 60 : 38) : (hs > 64 ? 44 : 24);
}

// Warps of a walker's team where rows are drafted tokens: as many as 16 pairs each of a sequence's pairs ask for, on average (a call's host
// side knows no more), up to 4.
__host__ __device__ inline int team_of(int B, int G, int n_heads, int n_kv_heads) {
    const long long pairs = (long long)B * cdiv(n_heads, n_kv_heads);
    return pairs <= 16ll * G ? 1 : pairs <= 32ll * G ? 2 : 4;
}

// Whether the tensor-core role takes a prefix of so many keys that serves n pairs of a KV head.  Its blocks start slower (8 us to
// the first parts where a walk has them after 4), so it takes what would keep the walkers for a while if all groups were alike:
// in 16-bit caches 10 us of them all, in fp32 ones 1 us, since their split products walk slower.  Over 60 calls of 1 to 64
// rows with prefixes of 16 to 12000, geometric means with no such limit and with this one: bf16 15.4 and 13.1 us, fp16 17.5 and 14.3;
// with a limit eight times higher, one of 64 rows and five prefixes of up to 16390 took 40 us instead of 32.
constexpr int kTcLeast16 = 40000, kTcLeast32 = 4000;
// In a tree's call teams of warps take up to 32 pairs (fp32: 64) faster: 217 us against 278 in the calls above (32 pairs, bf16; 64 pairs: 388, 312),
// in fp32 369 against 595 (64 pairs: 720, 706), and longer ones, too: 32 sequences of 300 to 600 keys, 64 pairs, 49 us against 62.
constexpr int kTreeTcLeast16 = 100000;
__host__ __device__ __forceinline__ bool tc_worth(const PagesAttn &p, int n, int keys) {
    return n > (!p.tree ? kM : p.dtype == 0 ? 64 : 32) && (long long)cdiv(n, kM) * p.n_kv_heads * p.G * tile_cost(p.dtype, kM) * (keys >> p.tile_shift) >=
                         (p.dtype == 0 ? kTcLeast32 : p.tree ? kTreeTcLeast16 : kTcLeast16);
}

// The last entry i of an ascending list of n (every `stride`-th int of a, the first at most x) that is at most x,
// found by a whole warp.
__device__ __forceinline__ int warp_find(const int *a, int stride, int n, int x) {
    int lo = 0, hi = n;
#pragma unroll 1
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, at = lo + (int)(threadIdx.x & 31) * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < hi && a[(size_t)(at < n ? at : n - 1) * stride] <= x);
        lo += (31 - __clz(m)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// key / page_size; page_shift is its logarithm where it is a power of two, else -1.
__device__ __forceinline__ int page_of(const PagesAttn &p, int key) {
    return p.page_shift >= 0 ? key >> p.page_shift : (int)((unsigned)key / (unsigned)p.page_size);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on) {
    const int n = on ? 16 : 0;  // 0: the 16 bytes are filled with zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One item's share of a walker's range, as the copying side hands it to the computing side (in shared memory).
struct alignas(16) WalkItem {
    int slot, n_tiles, left;          // item number of all, tiles, keys from the first tile on
    int row0, m0, pairs, head0, nh;   // rows, first pair, pairs, query heads head0 .. head0 + nh - 1 (trees: and 2^16 times the source's rows)
};
constexpr int ring_items(int team) { return team > 1 ? 16 : 8; }  // a ring of them a warp: more than the tiles, so the items, that copies are ahead

// The copies of a walking warp run through the tiles of its range in order, item after item, without a break: step()
// copies one tile and finds the next, whose page ids then have a tile's time to arrive.
// TEAM (trees): so many warps share a tile, the `member`-th copying its part of the rows; an item has kM pairs for each.  Their walks
// are the same.
template <int KT, int ROW, bool TREE, int TEAM = 1>
struct Walk {
    static constexpr int kPairs = kM * TEAM, kStart = item_cost(TREE, TEAM), kItems = ring_items(TEAM);
    const int *table;
    long long head;       // byte offset of the KV head
    int src, x, x1;       // source, cost up to which tiles are found, end of the range
    int rem, key, key1;   // tiles of the item not yet copied, this lane's key of the next one, end of the item's keys
    int page;             // page of that key
    int issued, items;    // tiles copied, items found
    bool on;

    __device__ __forceinline__ void start(const PagesAttn &p, const Plan &pl, int wid) {
        const int S = TREE ? p.G : p.G + p.B;
        const int T = pl.hdr[kHdrCost], per = pl.hdr[kHdrPer];
        x = min(wid * per, T);
        x1 = min(x + per, T);
        src = x < x1 ? warp_find(&pl.src[0].t0, sizeof(Source) / 4, S + 1, x) : 0;
        rem = issued = items = 0;
        on = x < x1;
    }

    // The item of the next tile that starts at x or after, in the range: into queue, its first tile next.
    __device__ __forceinline__ void find(const PagesAttn &p, const Plan &pl, int gq, WalkItem *queue) {
#pragma unroll 1
        for (;; ++src) {
            if (x >= x1) break;
            const int4 a = *reinterpret_cast<const int4 *>(&pl.src[src].t0), b = *reinterpret_cast<const int4 *>(&pl.src[src].key0);
            const int kt = a.z, cost = a.w, n = b.w * gq, tiles_m = (n + kPairs - 1) / kPairs;
            if (kt == 0) continue;
            x = max(x, a.x);
            const int len = kStart + kt * cost;
            int item = (int)((unsigned)(x - a.x) / (unsigned)len), at = a.x + item * len;  // item of the source, its place
            int k_first = x == at ? 0 : max(1, cdiv(max(x - at - kStart, 0), cost));
            if (k_first >= kt) {
                ++item;
                at += len;
                k_first = 0;
            }
            x = at + tile_place(k_first, kStart, cost);
            if (item >= tiles_m * p.n_kv_heads) continue;
            if (x >= x1) break;
            const int kvh = (int)((unsigned)item / (unsigned)tiles_m), m0 = (item - kvh * tiles_m) * kPairs;
            const int end = min(kt, max(k_first + 1, cdiv(max(x1 - at - kStart, 0), cost)));
            rem = end - k_first;
            x = end == kt ? at + len : at + tile_place(end, kStart, cost);
            key = b.x + k_first * KT;
            key1 = b.y;
            head = kvh * p.head_stride;
            table = p.table + (size_t)pl.src[src].seq * p.max_pages;
            if ((threadIdx.x & 31) == 0) {
                const int h0 = first_head(kvh, p.n_heads, p.n_kv_heads);
                int4 *q = reinterpret_cast<int4 *>(queue + items % kItems);
                q[0] = make_int4(a.y + item, rem, key1 - key, b.z);
                const int nh = first_head(kvh + 1, p.n_heads, p.n_kv_heads) - h0;
                q[1] = make_int4(m0, min(kPairs, n - m0), h0, TREE ? nh | b.w << 16 : nh);
            }
            key += threadIdx.x & 31;
            ++items;
            return;
        }
        on = false;
    }

    // Copies the next tile into the K and V regions at ks and vs of shared memory (16-byte word c of row r at word swz(r) ^ c;
    // rows past the item's end and words past the head are zeros) as one group, an empty one when there are no more; the
    // first call only finds the first.
    template <class Swz>
    __device__ __forceinline__ void step(const PagesAttn &p, const Plan &pl, int gq, int words, WalkItem *queue, uint32_t ks, uint32_t vs,
                                         Swz swz, int member = 0) {
        if (on) {
            if (rem) {
                constexpr int C = ROW / 16, RP = 32 / C;  // words a row, rows one instruction covers
                const int lane = threadIdx.x & 31, c = lane % C, rr = lane / C;
                // byte offset of this lane's row, -1 past the end or where the table is bad
                long long off = -1;
                if (lane < KT && key < key1) {
                    if (page >= 0 && page < p.n_pages)
                        off = head + page * p.page_stride + (key - page_of(p, key) * p.page_size) * p.row_stride;
                    else
                        atomicOr(p.err, L2_DEV_ERR_BOUNDS);
                }
#pragma unroll
                for (int r0 = 0; r0 < KT / TEAM; r0 += RP) {
                    const int r = (TEAM > 1 ? member * (KT / TEAM) : 0) + r0 + rr;
                    const long long o = __shfl_sync(0xffffffffu, off, r);
                    const bool in = o >= 0 && c < words;
                    const uint32_t d = r * ROW + ((c ^ swz(r)) << 4);
                    const long long so = in ? o + (c << 4) : 0;
                    cp_async16(ks + d, p.k + so, in);
                    cp_async16(vs + d, p.v + so, in);
                }
                ++issued;
                --rem;
                key += KT;
            }
            if (rem == 0) find(p, pl, gq, queue);
            page = on && (threadIdx.x & 31) < KT && key < key1 ? table[page_of(p, key)] : 0;
        }
        cp_commit();
    }
};

// The query of pair i of an item (row m / gq of the source, head m % gq of the KV head, m = m0 + i), or nullptr.
__device__ __forceinline__ const char *walk_query(const PagesAttn &p, const WalkItem &w, int i, int gq) {
    const int m = w.m0 + i, r = (int)((unsigned)m / (unsigned)gq), j = m - r * gq;
    return i < w.pairs && j < w.nh ? p.q + (w.row0 + r) * p.q_row + (w.head0 + j) * p.q_head : nullptr;
}

// What a walker knows of its item where rows are drafted tokens: how many the source has, and, in lane i, for pair i & 15, which of
// them its token sees, a bit each.  It sees all keys before theirs.
struct TreeItem {
    int n;
    u64 sees;
};
// The words are made where the item's last tile reaches the drafted rows.  w: the team's item, then its `member`-th warp's own pairs.
template <int KT>
__device__ __forceinline__ TreeItem tree_item(const PagesAttn &p, WalkItem &w, int gq, int member) {
    TreeItem t;
    t.n = w.nh >> 16;
    w.nh &= 0xffff;
    w.m0 += kM * member;
    w.pairs = max(0, min(kM, w.pairs - kM * member));
    t.sees = ~0ull;
    if (w.left - w.n_tiles * KT < t.n) {
        const TreeWords words = tree_words(tree_parents(p.parents ? p.parents + w.row0 : nullptr, t.n));
        const int m = w.m0 + (int)(threadIdx.x & 15);
        t.sees = tree_word(words, min((int)((unsigned)m / (unsigned)gq), kTreeNodes - 1));
    }
    return t;
}
// Keys of a tile that a token sees, bit k for key k: `left` keys from the tile's first to the end of the sequence, the last n of them drafted.
__device__ __forceinline__ unsigned tree_bits(u64 sees, int n, int left) {
    const int at = n - left;  // of the tile's first key among the drafted ones
    return at >= 0 ? (unsigned)(sees >> at) : at <= -32 ? ~0u : (unsigned)(sees << -at) | ((1u << -at) - 1u);
}

// Waits for the warps of a team (number `team` of its block's).
template <int TEAM>
__device__ __forceinline__ void team_sync(int team) {
    if constexpr (TEAM == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * TEAM) : "memory");
}

// Walkers that are warps: neighbours in the numbering sit in different blocks, so that a stretch of costlier tiles
// does not fall on one SM.  warp: of the block's walking ones; block0: the first walking block.
__device__ __forceinline__ int walker_id(int warp, int block0) { return warp * (gridDim.x - block0) + blockIdx.x - block0; }

}  // namespace l2
