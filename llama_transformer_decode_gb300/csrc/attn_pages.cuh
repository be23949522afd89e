// What the kernels of the paged attention share: the plan in the workspace and the numbering of the
// parts they leave for the merge.
#pragma once
#include <cstddef>
#include <cuda_runtime.h>

#include "l2_pages.h"

namespace l2 {

constexpr int kM = 16;      // (row, head) pairs of a warp's item
constexpr int kTcKeys = 128;  // keys of a tensor-core tile
constexpr int kTcRows = 128;  // pairs of a tensor-core slot; an item has up to two slots' worth

// Plan: a header; per source of the warps (S = G + B) its first tile, first item, tiles per item, key range and
// rows; per group, for the tensor-core kernel, its first tile, tiles per item and first row of its parts.
enum { kHdrTiles = 0, kHdrWarps = 1, kHdrOk = 2, kHdrTcTiles = 3, kHdrTcCtas = 4, kHdrInts = 16 };
struct Plan {
    int *hdr, *t0, *i0, *kt, *key0, *key1, *row0, *rows;
    int *tc_t0, *tc_kt, *tc_r0;
};
__host__ __device__ inline Plan plan_of(int *base, int S, int G) {
    Plan p;
    p.hdr = base;
    p.t0 = base + kHdrInts;
    p.i0 = p.t0 + S + 1;
    p.kt = p.i0 + S + 1;
    p.key0 = p.kt + S;
    p.key1 = p.key0 + S;
    p.row0 = p.key1 + S;
    p.rows = p.row0 + S;
    p.tc_t0 = p.rows + S;
    p.tc_kt = p.tc_t0 + G + 1;
    p.tc_r0 = p.tc_kt + G;
    return p;
}
__host__ __device__ inline size_t plan_ints(int S, int G) {
    return (kHdrInts + 2 * (size_t)(S + 1) + 5 * (size_t)S + 3 * (size_t)G + 1 + 63) / 64 * 64;
}

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Most query heads of a KV head; head j of KV head g is first_head(g) + j.
__host__ __device__ __forceinline__ int heads_per_kv(int H, int KV) { return (H + KV - 1) / KV; }
__device__ __forceinline__ int first_head(int g, int H, int KV) { return (g * H + KV - 1) / KV; }

// T tiles are cut evenly over W walkers: walker w takes tiles [first_of(w), first_of(w + 1)).
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

// The last entry i of an ascending list a[0 .. n) (a[0] <= x) with a[i] <= x, found by a whole warp.
__device__ __forceinline__ int warp_find(const int *a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = cdiv(hi - lo, 32), at = lo + (int)(threadIdx.x & 31) * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < hi && a[at < n ? at : n - 1] <= x);
        lo += (31 - __clz(m)) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    return lo;
}

}  // namespace l2
