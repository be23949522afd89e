// What the kernels of the paged attention share: the plan in the workspace and the numbering of the
// parts they leave for the merge.
#pragma once
#include <cstddef>
#include <cuda_runtime.h>

#include "l2_pages.h"

namespace l2 {

constexpr int kM = 16;         // (row, head) pairs of a warp's item
constexpr int kTcRows = 128;  // pairs of a tensor-core slot; an item has up to two slots' worth

// Plan: a header; the sources of the warps (the groups' prefixes, then the rows' own keys: S = G + B, and an end);
// per group, for the tensor-core role, the cost before it, tiles per item and first row of its parts; the group of
// each row.
enum { kHdrCost = 0, kHdrWarps = 1, kHdrOk = 2, kHdrTcCost = 3, kHdrTcBlocks = 4, kHdrInts = 16 };
struct alignas(16) Source {
    int t0, i0, kt, cost;          // cost and items of the sources before it, tiles per item, cost of a tile
    int key0, key1, row0, rows;    // keys, rows
    int seq, pad[3];               // sequence whose table finds the keys
};
struct Plan {
    int *hdr;
    Source *src;
    int *tc_t0, *tc_kt, *tc_r0, *group;
};
__host__ __device__ inline Plan plan_of(void *base, int B, int G) {
    Plan p;
    p.hdr = static_cast<int *>(base);
    p.src = reinterpret_cast<Source *>(p.hdr + kHdrInts);
    p.tc_t0 = reinterpret_cast<int *>(p.src + G + B + 1);
    p.tc_kt = p.tc_t0 + G + 1;
    p.tc_r0 = p.tc_kt + G;
    p.group = p.tc_r0 + G;
    return p;
}
__host__ __device__ constexpr size_t plan_bytes(int B, int G) {
    return (kHdrInts * 4 + (size_t)(G + B + 1) * sizeof(Source) + (3 * (size_t)G + 1 + B) * 4 + 127) / 128 * 128;
}
// A call of at most this many sources is planned by every block of its kernels for itself, in shared memory: about
// 2 us of latency where a kernel of its own before them costs 6.  Larger calls have such a kernel.
constexpr int kPlanInBlock = 192;
constexpr size_t kPlanSmem = plan_bytes(kPlanInBlock / 2, kPlanInBlock / 2);  // the most for G + B sources, G <= B

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Most query heads of a KV head; head j of KV head g is first_head(g) + j.
__host__ __device__ __forceinline__ int heads_per_kv(int H, int KV) { return (H + KV - 1) / KV; }
__device__ __forceinline__ int first_head(int g, int H, int KV) { return (g * H + KV - 1) / KV; }

// T tiles (or units of cost) are cut evenly over W walkers: walker w takes [first_of(w), first_of(w + 1)).
__device__ __forceinline__ int first_of(int w, int T, int W) { return (int)((long long)w * T / W); }
__device__ __forceinline__ int walker_of(int tile, int T, int W) { return (int)((((long long)tile + 1) * W + T - 1) / T - 1); }

// Tensor-core items of a group: n pairs (row, head) of one KV head in runs of up to 256.  A run of up to 128
// pairs is served by both slots, which take alternate tiles and leave a part of n rows each; of a
// longer one slot 0 takes the first 128.  Parts of walker w and a run: rows
// tc_r0 + (rows of the group's runs before) + 256 w of the parts' arrays, which keeps
// them apart: from walker to walker by 256 rows, from run to run by the run's own.
__host__ __device__ __forceinline__ int tc_runs(int n) { return cdiv(n, 2 * kTcRows); }
__host__ __device__ __forceinline__ int tc_run_rows(int n) { return n > kTcRows ? n : 2 * n; }
__host__ __device__ __forceinline__ int tc_head_rows(int n) {  // of all runs of one KV head
    const int full = tc_runs(n) - 1;
    return 2 * kTcRows * full + tc_run_rows(n - 2 * kTcRows * full);
}

// Walkers that are warps: neighbours in the numbering sit in different blocks, so that a stretch of costlier tiles
// does not fall on one SM.
__device__ __forceinline__ int walker_id(int warp, int block0) { return warp * (gridDim.x - block0) + blockIdx.x - block0; }

// The last entry i of an ascending list of n (every `stride`-th int of a, the first at most x) that is at most x,
// found by a whole warp.
__device__ __forceinline__ int warp_find(const int *a, int stride, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = cdiv(hi - lo, 32), at = lo + (int)(threadIdx.x & 31) * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < hi && a[(size_t)(at < n ? at : n - 1) * stride] <= x);
        lo += (31 - __clz(m)) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    return lo;
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

// Cost of a tile of an item of n pairs, in quarters of reading it.  16-bit: reading bounds every size.  fp32 FMAs take
// over from 8 pairs on; measured on GB300, 1 GB of suffixes of head size 128 / 64: 166 / 167 us at 1 pair, 174 / 167 at
// 4, 198 / 198 at 8, 271 / 279 at 16.
constexpr int kCostUnit = 4;
__host__ __device__ __forceinline__ int tile_cost(int dtype, int n) { return dtype != 0 || n <= 4 ? 4 : n <= 8 ? 5 : 7; }

// Cost of a tensor-core tile for n pairs of a KV head, in the same unit (a quarter of 8 KB): reading its 32 KB while the
// slots take turns, the slots' time when both work on every tile.
__host__ __device__ __forceinline__ int tc_cost(int n, int hs) { return n > kTcRows ? 28 : 16; }

// key / page_size; page_shift is its logarithm where it is a power of two, else -1.
__device__ __forceinline__ int page_of(const PagesAttn &p, int key) {
    return p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
}

// One item's share of a walker's range, for the kernels whose walkers are warps.
struct WalkItem {
    int item, slot, k_first, n_tiles;          // item within its source and of all, tiles k_first .. k_first + n_tiles - 1
    int row0, key0, key1, head0, nh, kvh, m0;  // rows, keys, query heads head0 .. head0 + nh - 1, first pair
    int pairs;                                 // pairs of the item
    const int *table;                          // page table its keys are found through
};
// The item whose tile starts at cost x or next after it (a tile belongs to the walker in whose range it starts),
// and the tiles of it that start before x1; x moves behind them, src past finished sources.  False: no more.
__device__ __forceinline__ bool walk_item(const PagesAttn &p, const Plan &pl, int &src, int &x, int x1, int gq, WalkItem &w) {
    for (;; ++src) {
        if (x >= x1) return false;
        const int4 a = *reinterpret_cast<const int4 *>(&pl.src[src].t0), b = *reinterpret_cast<const int4 *>(&pl.src[src].key0);
        const int kt = a.z, cost = a.w, n = b.w * gq, tiles_m = cdiv(n, kM);
        if (kt == 0) continue;
        const int i = cdiv(x - a.x, cost);  // tile of the source
        x = a.x + i * cost;
        w.item = i / kt;
        if (w.item >= tiles_m * p.n_kv_heads) continue;
        if (x >= x1) return false;
        w.slot = a.y + w.item;
        w.k_first = i - w.item * kt;
        w.n_tiles = min(kt - w.k_first, cdiv(x1 - x, cost));
        x += w.n_tiles * cost;
        w.row0 = b.z;
        w.key0 = b.x;
        w.key1 = b.y;
        w.kvh = w.item / tiles_m;
        w.m0 = (w.item - w.kvh * tiles_m) * kM;
        w.pairs = min(kM, n - w.m0);
        w.head0 = first_head(w.kvh, p.n_heads, p.n_kv_heads);
        w.nh = first_head(w.kvh + 1, p.n_heads, p.n_kv_heads) - w.head0;
        w.table = p.table + (size_t)pl.src[src].seq * p.max_pages;
        return true;
    }
}
// The query of pair m (row m / gq of the source, head m % gq of the KV head), or nullptr.
__device__ __forceinline__ const char *walk_query(const PagesAttn &p, const WalkItem &w, int i, int gq) {
    const int m = w.m0 + i, r = m / gq, j = m - r * gq;
    return i < w.pairs && j < w.nh ? p.q + (w.row0 + r) * p.q_row + (w.head0 + j) * p.q_head : nullptr;
}
// A key's row is found in two steps, so that the load of the table entry is a tile old when its value is first
// looked at: the page of `key` (0 past the item's end), and then the byte offset of the row in its KV head's pages, or
// -1 past the end or where the table is bad.
__device__ __forceinline__ int walk_page(const PagesAttn &p, const WalkItem &w, int key) {
    return key < w.key1 ? w.table[page_of(p, key)] : 0;
}
__device__ __forceinline__ long long walk_place(const PagesAttn &p, const WalkItem &w, int key, int page) {
    if (key >= w.key1) return -1;
    if (page < 0 || page >= p.n_pages) {
        atomicOr(p.err, L2_DEV_ERR_BOUNDS);
        return -1;
    }
    return page * p.page_stride + (key - page_of(p, key) * p.page_size) * p.row_stride;
}


// The tiles of a walker's whole range in order, one ahead of the copies: the next tile's key of this lane and its page, whose
// load has a tile's time to return.  The copies run through the items without a break, so a new item's first tiles are in
// flight while the one before is computed.
template <int KT>
struct WalkAhead {
    WalkItem w;
    int src, x, i, key, page;
    bool on;
    __device__ __forceinline__ void look(const PagesAttn &p) {
        const int lane = threadIdx.x & 31;
        key = on && lane < KT ? w.key0 + (w.k_first + i) * KT + lane : w.key1;
        page = on ? walk_page(p, w, key) : 0;
    }
    __device__ __forceinline__ void start(const PagesAttn &p, const Plan &pl, int src0, int x0, int x1, int gq) {
        src = src0;
        x = x0;
        i = 0;
        on = walk_item(p, pl, src, x, x1, gq, w);
        look(p);
    }
    __device__ __forceinline__ void next(const PagesAttn &p, const Plan &pl, int x1, int gq) {
        if (++i >= w.n_tiles) {
            i = 0;
            on = walk_item(p, pl, src, x, x1, gq, w);
        }
        look(p);
    }
};

// Copies the next tile into the K and V regions at ks and vs of shared memory (rows of ROW bytes, 16-byte word c of row r
// at word swz(r) ^ c; rows past the item's end and words past the head are zeros) as one group; none when there are no more.
template <int KT, int ROW, class Swz>
__device__ __forceinline__ void walk_copy(const PagesAttn &p, const Plan &pl, WalkAhead<KT> &a, int x1, int gq, int words,
                                          uint32_t ks, uint32_t vs, Swz swz) {
    if (a.on) {
        constexpr int C = ROW / 16, RP = 32 / C;  // words a row, rows one instruction covers
        const int lane = threadIdx.x & 31, c = lane % C, rr = lane / C;
        const long long off = walk_place(p, a.w, a.key, a.page);
        const char *kb = p.k + a.w.kvh * p.head_stride, *vb = p.v + a.w.kvh * p.head_stride;
#pragma unroll
        for (int r0 = 0; r0 < KT; r0 += RP) {
            const int r = r0 + rr;
            const long long o = __shfl_sync(0xffffffffu, off, r);
            const bool on = o >= 0 && c < words;
            const uint32_t d = r * ROW + ((c ^ swz(r)) << 4);
            const long long so = on ? o + (c << 4) : 0;
            cp_async16(ks + d, kb + so, on);
            cp_async16(vs + d, vb + so, on);
        }
        a.next(p, pl, x1, gq);
    }
    cp_commit();
}

}  // namespace l2
