// The plan of a paged attention call: lengths of the sources and the numbering of their tiles and items.  Built by one
// block of NT threads, either a kernel of its own or, for calls of few sources, every block of the kernels for itself.
#pragma once
#include "attn_pages.cuh"

namespace l2 {

// Fewest tiles a warp takes: below that the parts cost more to write and merge than the parallel reading gains.
constexpr int kMinTiles = 4;
constexpr int kTcMinTiles = 2;  // the same for the blocks of the tensor-core role

template <int NT, int MAX>
struct PlanScratch {
    int minlen[MAX], mintc[MAX], gstart[MAX + 1], len[MAX], group[MAX], seq[MAX];
    long long sums[2][NT / 32];
};

// Exclusive prefix sums over the block of the low and the high 32 bits (both sums below 2^31), and the totals.
template <int NT>
__device__ __forceinline__ long long plan_scan(long long v, long long *total, long long *buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) buf[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const long long t = buf[w];
        before += w < warp ? t : 0;
        all += t;
    }
    *total = all;
    return before + x - v;
}

// MAX: most groups or rows (MAX <= NT).  Ends with a barrier.  report: sets the status word when the call is bad.
template <int NT, int MAX>
__device__ __forceinline__ void plan_build(const PagesAttn &p, const Plan &pl, PlanScratch<NT, MAX> &sc, bool report) {
    const int i = threadIdx.x, S = p.G + p.B, gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    bool bad = false;
    int len = 0, seq = 0, P = 0, a0 = 0;
    // what depends on nothing is loaded before the lengths, which depend on seqs
    if (i < p.G) P = p.prefix_lens[i];
    if (p.G && i <= p.G) a0 = p.group_starts[i];
    if (i < p.B) {
        seq = p.seqs ? p.seqs[i] : i;
        bad = seq < 0 || seq >= p.n_seqs;
        if (!bad) len = p.lens[seq];
        bad |= len < 0 || len > (long long)p.max_pages * p.page_size;
        sc.len[i] = len;
        sc.seq[i] = seq;
    }
    if (p.G) {
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
    if (__syncthreads_or(bad)) {
        if (i == 0) {
            if (report) atomicOr(p.err, L2_PAGES_ERR_ARGS);
            pl.hdr[kHdrCost] = pl.hdr[kHdrTcCost] = pl.hdr[kHdrTcBlocks] = 0;
            pl.hdr[kHdrWarps] = 1;
            pl.hdr[kHdrOk] = 0;
        }
        __syncthreads();
        return;
    }
    long long tc_all = 0;
    if (p.G) {
        if (i < p.B) {
            int lo = 0, hi = p.G;  // the group of the row: the last that starts at or before it
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                sc.gstart[m] <= i ? lo = m : hi = m;
            }
            atomicMin(&sc.minlen[lo], len);
            sc.group[i] = pl.group[i] = lo;
        }
        __syncthreads();
        // prefixes worth it go to the tensor cores in whole tiles of 128 keys; what is left of them stays with the warps
        const int n = i < p.G ? (sc.gstart[i + 1] - sc.gstart[i]) * gq : 0, full = i < p.G && p.tc && n > kM ? sc.minlen[i] / p.tc_keys : 0;
        const int tiles = full * tc_runs(n) * p.n_kv_heads * tc_cost(n, p.head_size), prows = full ? tc_head_rows(n) * p.n_kv_heads : 0;
        const long long before = plan_scan<NT>((long long)tiles << 32 | prows, &tc_all, sc.sums[0]);
        if (i < p.G) {
            pl.tc_t0[i] = (int)(before >> 32);
            pl.tc_kt[i] = full;
            pl.tc_r0[i] = (int)before;
            sc.mintc[i] = full * p.tc_keys;
        }
        __syncthreads();
    }
    long long all = 0;
    for (int s0 = 0; s0 < S; s0 += NT) {
        const int s = s0 + i;
        Source e = {};
        if (s < p.G) {
            e.key0 = sc.mintc[s];
            e.key1 = sc.minlen[s];
            e.row0 = sc.gstart[s];
            e.rows = sc.gstart[s + 1] - e.row0;
        } else if (s < S) {
            e.row0 = s - p.G;
            e.rows = 1;
            e.key0 = p.G ? sc.minlen[sc.group[e.row0]] : 0;
            e.key1 = sc.len[e.row0];
        }
        e.kt = s < S ? cdiv(e.key1 - e.key0, p.tile_keys) : 0;
        if (s < p.G ? e.rows > 0 : s < S) e.seq = sc.seq[e.row0];
        e.cost = tile_cost(p.dtype, min(e.rows * gq, kM));
        const int items = e.kt ? cdiv(e.rows * gq, kM) * p.n_kv_heads : 0;
        long long here;
        const long long before = all + plan_scan<NT>((long long)(items * e.kt * e.cost) << 32 | items, &here, sc.sums[1]);
        e.t0 = (int)(before >> 32);
        e.i0 = (int)before;
        if (s < S) pl.src[s] = e;
        all += here;
        if (s0 + NT < S) __syncthreads();
    }
    if (i == 0) {
        const int cost = (int)(all >> 32), tc = (int)(tc_all >> 32);
        // blocks of the two roles by cost, at least one of each that has work
        int n_tc = 0;
        if (tc) {
            n_tc = (int)(((long long)tc * p.num_sms + (tc + (long long)cost) / 2) / (tc + (long long)cost));
            n_tc = max(1, min(min(n_tc, cdiv(tc, kTcMinTiles * tc_cost(1, p.head_size))), p.num_sms - (cost ? 1 : 0)));
        }
        pl.src[S].t0 = cost;
        pl.hdr[kHdrCost] = cost;
        pl.hdr[kHdrWarps] = max(1, min((p.num_sms - n_tc) * p.walk_warps, cdiv(cost, kMinTiles * kCostUnit)));
        pl.hdr[kHdrTcCost] = tc;
        pl.hdr[kHdrTcBlocks] = n_tc;
        if (p.G) pl.tc_t0[p.G] = tc;
        pl.hdr[kHdrOk] = 1;
    }
    __syncthreads();
}

// The plan as a kernel's block uses it: built here (mem: kPlanSmem bytes, scratch: free until the caller's first
// use of it; `keep`: also left in the workspace for the merge), or the workspace's.
template <int NT>
__device__ __forceinline__ Plan plan_here(const PagesAttn &p, void *mem, void *scratch, bool keep) {
    const Plan out = plan_of(p.plan, p.B, p.G);
    if (!p.plan_in_block) return out;
    const Plan pl = plan_of(mem, p.B, p.G);
    plan_build<NT, kPlanInBlock>(p, pl, *static_cast<PlanScratch<NT, kPlanInBlock> *>(scratch), keep);
    if (keep)
        for (int i = threadIdx.x; i < (int)(plan_bytes(p.B, p.G) / 4); i += NT) p.plan[i] = static_cast<const int *>(mem)[i];
    return pl;
}

}  // namespace l2
