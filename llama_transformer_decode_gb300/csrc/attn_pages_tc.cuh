// The shared prefixes of the paged attention on the tensor cores (16-bit caches): one role of the blocks of
// attn_pages_16.cu.
//
// What it computes: the parts (m, l, acc) of attn_pages.cu for the whole 128-key tiles of each
// prefix, for all (row, query head) pairs of the group and KV head at once: S = Q K^T, weights
// P = 2^(x - m), acc = P V, with pairs as the M of tcgen05.mma, keys as N of the first product and K of
// the second.
//
// How.  An item is a KV head and a run of up to 256 pairs; all (item, tile) steps are split by cost over
// the blocks that take this role.  A block has two slots, each with 128 lanes of scores and of acc in tensor
// memory and four softmax warps: a run of more than 128 pairs gives each slot half of the pairs and the
// same tiles (K and V are read once for 256 pairs); a shorter run goes to both slots, which
// take alternate tiles, so that one slot's softmax runs beside the other's products.
//   warp 0     tiles of K and V by TMA into two rings (128-byte swizzle; a box is a page's rows
//              that fall into the tile, so pages of 8, 16, 32, 64 rows or a multiple of 128 are gathered
//              without a copy); rows past the prefix are never loaded, so nothing is masked
//   warps 1-2  the products of slots 0 and 1
//   warps 4-7, 8-11  slots 0 and 1: queries to shared memory, softmax, parts out
// A thread owns one pair: its row of scores is a lane of tensor memory, so max and sum need no
// exchange.  The weights go back over the scores as sums of two 16-bit values, which is what the walk of attn_pages_16.cu takes (off by at
// most 2^-16 of a weight in bf16, 2^-22 in fp16), and are the A operand of the second product from there, once for each; the sums l are
// of the fp32 weights.  acc is rescaled only when a row's maximum has grown by more than a factor of 2^kGrow since the
// last time.  In bf16 weights then stay below 2^8.  fp16 ends at 2^16 and its least step is 2^-24, so its weights are
// 2^(x - m + 13), at most 2^15: rounding then loses at most 2^-38 of the largest weight on each, where without the 13
// a prefix of 131072 keys whose weights are 2^-26 of one other key's lost a 512th of the sum.  (One value a weight took 101 us in
// place of 108 for 32 KV heads of 64 pairs and 16384 bf16 keys, and left an error of 0.0023 in place of 0.0017 against 64 bits, the latter
// what rounding the exact output leaves; how many bits a row got then hung on what else was in its call.)  The second product
// of a tile's first 64 keys is issued while the weights of the others are made (256 pairs of head size 128: 4.1 -> 3.2 us a tile).
//
// What bounds it: up to 128 pairs, reading K and V; above, the products, the exponentials and the cutting of
// the weights, one after the other for each slot.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "attn_pages.cuh"
#include "attn_plan.cuh"
#include "attn_slots.h"
#include "l2_device.cuh"
#include "l2_pages.h"
#include "l2_tc.cuh"

namespace l2 {

namespace {

constexpr int kSlotThreads = 128;
constexpr int kRing = 4;                    // most stages of a ring
// See above: a row's weights are at most 2^(lift + grow) of its type.
template <bool BF>
constexpr float kLiftTc = BF ? 0.f : 13.f;
template <bool BF>
constexpr float kGrow = BF ? 8.f : 2.f;

struct alignas(128) TcAttn {
    CUtensorMap kmap, vmap;
    PagesAttn p;
    int box_rows;
    float scale_log2;  // positive; the queries carry its sign
    uint32_t flip;     // 0x8000 in both halves when the scale is negative
};

// Tensor memory of slot s, columns from 256 s on: scores, then, in their place, weights as 16-bit pairs (of 64 keys at a time the 32
// columns of the larger values, then those of what they leave), and acc from kO on.  The next scores wait for the product that reads
// the weights.  (Tiles of 64 keys, which would leave room for the scores beside them, were slower: 215 us against 152 for 65408
// keys, 8 KV heads and 512 pairs each.)
template <int HS>
struct TcShape {
    static constexpr int KT = tc_keys(false);
    static constexpr int kBlocks = HS / 64;                  // 64-value blocks of a row
    static constexpr uint32_t kBlock = KT * 128, kQBlock = kTcRows * 128;
    static constexpr uint32_t kTile = kBlocks * kBlock, kQ = kBlocks * kQBlock;
    static constexpr int kStages = HS == 64 ? 4 : 2;         // of each ring
    static constexpr uint32_t kTiles = 2 * kQ + 2 * kStages * kTile;
    static constexpr uint32_t kSmem = 1024 + 1024 + kTiles;  // alignment, barriers
    static constexpr int kO = KT;
    static_assert(kO + HS <= 256, "a slot has 256 columns");
};

struct TcFx {
    uint64_t full_k[kTakers][kRing], empty_k[kRing], full_v[kTakers][kRing], empty_v[kRing];  // full: by who takes the tile
    uint64_t q_full[2], s_full[2], p_half[2], p_full[2], pv_done[2], fin[2];
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(TcFx) <= 1024, "the fixed block must fit before the tiles");

__device__ __forceinline__ void tensor4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

template <class Fx>
__device__ __forceinline__ bool stopped(const Fx &fx) { return *reinterpret_cast<const volatile int *>(&fx.abort) != 0; }
template <class Fx>
__device__ __forceinline__ void stop(Fx &fx) { *reinterpret_cast<volatile int *>(&fx.abort) = 1; }

// A bounded wait that also ends when another warp gave up; false: leave.
template <class Fx>
__device__ __forceinline__ bool wait_or_stop(Fx &fx, uint64_t *bar, uint32_t parity, int *err) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;  // the timer is read once the wait is long
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (stopped(fx)) return false;
        if ((i & 255u) == 0) {
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) {
                atomicOr(err, L2_DEV_ERR_TIMEOUT);
                stop(fx);
                return false;
            }
        }
    }
}

// D fp32, A (K-major) and B 16-bit; b_mn: B's contiguous dimension is N.
__device__ __forceinline__ uint32_t idesc_f16(bool bf, int M, int N, bool b_mn) {
    return (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 2^x, at most 2 units in the last place off; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One item's part of a block's range of steps.
struct Seg {
    int group, kvh, m0, rows, k0, n;  // m0: first pair, rows: pairs (up to 256), tiles k0 .. k0 + n - 1
    int out;                          // first row of its parts
};

// The next segment of block bid's range of cost, which ends at x_end: the tiles of one item that start in it, from x
// and group grp on.  Every warp of a block walks the same segments.
template <bool F32>
__device__ __forceinline__ bool tc_segment(const PagesAttn &p, const Plan &pl, int gq, int bid, int x_end, int &x, int &grp, Seg &g) {
#pragma unroll 1
    for (;; ++grp) {
        if (x >= x_end) return false;
        const int kt = pl.tc_kt[grp], t0 = pl.tc_t0[grp];
        if (kt == 0) continue;
        const int n = pl.src[grp].rows * gq, runs = tc_runs(n, F32), cost = tc_cost(n, p.head_size, F32), len = kTcItemCost + kt * cost;
        x = max(x, t0);
        int item = (int)((unsigned)(x - t0) / (unsigned)len), at = t0 + item * len;
        int k0 = x == at ? 0 : max(1, cdiv(max(x - at - kTcItemCost, 0), cost));
        if (k0 >= kt) {
            ++item;
            at += len;
            k0 = 0;
        }
        x = at + tile_place(k0, kTcItemCost, cost);
        if (item >= runs * p.n_kv_heads) continue;
        if (x >= x_end) return false;
        const int end = min(kt, max(k0 + 1, cdiv(max(x_end - at - kTcItemCost, 0), cost)));
        x = end == kt ? at + len : at + tile_place(end, kTcItemCost, cost);
        g.group = grp;
        g.kvh = (int)((unsigned)item / (unsigned)runs);
        const int run = item - g.kvh * runs;
        g.m0 = run * tc_run(F32);
        g.rows = min(tc_run(F32), n - g.m0);
        g.k0 = k0;
        g.n = end - k0;
        g.out = pl.tc_r0[grp] + g.kvh * tc_head_rows(n, F32) + g.m0 + tc_run(F32) * bid;
        return true;
    }
}

template <bool BF>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
    if constexpr (BF) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

template <bool BF>
__device__ __forceinline__ float2 unpack16(uint32_t v) {
    if constexpr (BF)
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// One block's work, all of its threads.  smem: kSmem bytes; pl: the plan; bid: the block among those of the role.
template <int HS, bool BF>
__device__ __forceinline__ void tc_role(const TcAttn &ta, const Plan &pl, unsigned char *smem_raw, int bid) {
    using Sh = TcShape<HS>;
    const PagesAttn &p = ta.p;
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    TcFx &fx = *reinterpret_cast<TcFx *>(smem);
    unsigned char *qs = smem + 1024;
    const uint32_t q_at = smem_u32(qs), k_at = q_at + 2 * Sh::kQ, v_at = k_at + Sh::kStages * Sh::kTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            for (int taker = 0; taker < kTakers; ++taker) {
                mbar_init(&fx.full_k[taker][i], 1);
                mbar_init(&fx.full_v[taker][i], 1);
            }
            mbar_init(&fx.empty_k[i], 2);  // a release by each slot
            mbar_init(&fx.empty_v[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&fx.q_full[i], kSlotThreads);
            mbar_init(&fx.s_full[i], 1);
            mbar_init(&fx.p_half[i], kSlotThreads);
            mbar_init(&fx.p_full[i], kSlotThreads);
            mbar_init(&fx.pv_done[i], 1);
        }
        mbar_init(&fx.fin[0], 1);
        mbar_init(&fx.fin[1], 1);
        fence_barrier_init();
        fx.abort = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&fx.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_proxy_async_smem();  // the plan was built over the rings' memory
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = fx.tmem;
    const int x_begin = bid * pl.hdr[kHdrTcPer], x_end = min(x_begin + pl.hdr[kHdrTcPer], pl.hdr[kHdrTcCost]);
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    auto segment = [&](int &x, int &grp, Seg &g) { return tc_segment<false>(p, pl, gq, bid, x_end, x, grp, g); };
    // tiles slot s works on
    auto slot_tiles = [&](const Seg &g, int s) { return g.rows > kTcRows ? g.n : (g.n + 1 - s) >> 1; };
    const int grp0 = x_begin < x_end ? warp_find(pl.tc_t0, 1, p.G + 1, x_begin) : 0;

    if (warp == 0) {
        // ---------------- copies: lane j issues box j of a tile ----------------
        int t = 0, grp = grp0;
        const int boxes = Sh::KT / ta.box_rows;
        bool ok = true;
        int x = x_begin;
        Seg g;
        while (ok && segment(x, grp, g)) {
            const int *table = p.table + (size_t)pl.src[g.group].seq * p.max_pages;
            auto lookup = [&](int tile) {
                const int pos = (g.k0 + tile) * Sh::KT + lane * ta.box_rows;
                return lane < boxes && tile < g.n ? table[page_of(p, pos)] : 0;
            };
            // one tile of K or V; its page ids were loaded a step before
            auto copy = [&](int kv, int tile, int tt, int page) {
                const int ns = Sh::kStages, st = tt % ns, taker = taker_of(tile, g.rows > kTcRows);
                uint64_t *full = kv ? &fx.full_v[taker][st] : &fx.full_k[taker][st], *empty = kv ? &fx.empty_v[st] : &fx.empty_k[st];
                if (tt >= ns) ok = wait_or_stop(fx, empty, (uint32_t)((tt / ns - 1) & 1), p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                if (lane == 0) mbar_arrive_expect_tx(full, Sh::kTile);
                __syncwarp();
                if (lane < boxes) {
                    const int pos = (g.k0 + tile) * Sh::KT + lane * ta.box_rows, row = pos - page_of(p, pos) * p.page_size;
                    const int cp = page >= 0 && page < p.n_pages ? page : p.n_pages;  // out of range: TMA fills zeros
                    if (cp == p.n_pages) atomicOr(p.err, L2_DEV_ERR_BOUNDS);
                    const uint32_t dst = (kv ? v_at : k_at) + st * Sh::kTile + lane * ta.box_rows * 128;
#pragma unroll
                    for (int b = 0; b < Sh::kBlocks; ++b) tensor4d(dst + b * Sh::kBlock, kv ? &ta.vmap : &ta.kmap, 64 * b, row, g.kvh, cp, full);
                }
                __syncwarp();
            };
            // K runs a tile ahead of V: its stage is free first, and a tile's scores are the first thing needed
            int pk = lookup(0), pn = lookup(1), pv = pk;
            for (int i = 0; i <= g.n && ok; ++i) {
                if (i < g.n) copy(0, i, t + i, pk);
                if (ok && i > 0) copy(1, i - 1, t + i - 1, pv);
                pv = pk;
                pk = pn;
                pn = lookup(i + 2);
            }
            t += g.n;
        }
        // the last stages' releases land before the block's memory goes; copies in flight do where something gave up
        for (int tt = max(0, t - Sh::kStages); tt < t && ok; ++tt) {
            const int st = tt % Sh::kStages;
            ok = wait_or_stop(fx, &fx.empty_k[st], (uint32_t)((tt / Sh::kStages) & 1), p.err) &&
                 wait_or_stop(fx, &fx.empty_v[st], (uint32_t)((tt / Sh::kStages) & 1), p.err);
        }
        if (!ok) {
            for (int st = 0; st < Sh::kStages; ++st)
                for (int w = 0; w < 2 * kTakers; ++w) {
                    (void)mbar_wait_limit(&fx.full_k[w >> 1][st], w & 1, p.err, 1000000ull);
                    (void)mbar_wait_limit(&fx.full_v[w >> 1][st], w & 1, p.err, 1000000ull);
                }
        }
    } else if (warp <= 2) {
        // ---------------- products: a warp per slot ----------------
        // The whole warp keeps the books, with values every lane shares (a shuffle from lane 0 tells the compiler so), and one
        // lane issues: descriptors then stay in uniform registers.  (Issued from inside a one-lane branch, a tile's twelve products
        // took 0.74 us; one warp for both slots let each slot wait behind the other's issue: 2.6 us a tile at head size 128.)
        const int s = warp - 1;
        auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
        bool ok = true;
        auto await = [&](uint64_t *bar, int parity) {
            ok = __all_sync(0xffffffffu, wait_or_stop(fx, bar, (uint32_t)parity & 1u, p.err));
            return ok;
        };
        const uint32_t tm = (uint32_t)uniform((int)tmem) + 256 * s;
        const uint32_t id_qk = idesc_f16(BF, kTcRows, Sh::KT, false), id_pv = idesc_f16(BF, kTcRows, HS, true);
        int grp = grp0, t_base = 0, x = x_begin, n_p = 0, nq = 0;  // tiles before the item, second products, items with tiles
        bool both = false;                                         // this item's tiles go to both slots
        Phases<Sh::kStages> k_phases, v_phases;
        // a tile's stage, and whether it has landed there
        auto see = [&](uint64_t (*full)[kRing], Phases<Sh::kStages> &phases, int tile) {
            const int st = tile % Sh::kStages, taker = taker_of(tile - t_base, both);
            return await(&full[taker][st], phases.next(taker, st));
        };
        auto see_k = [&](int tile) { return see(fx.full_k, k_phases, tile); };
        auto see_v = [&](int tile) { return see(fx.full_v, v_phases, tile); };
        auto queries = [&]() { return await(&fx.q_full[s], nq++); };
        auto scores = [&](int tile) {
            const int st = uniform(tile) % Sh::kStages;
            tc_fence_after();
            const uint64_t dq = desc_sw128(q_at + s * Sh::kQ), dk = desc_sw128(k_at + st * Sh::kTile);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < HS / 16; ++k)  // 32 bytes a step, blocks of 4 steps
                    mma_bf16(tm, dq + (uint64_t)(((k >> 2) * Sh::kQBlock + (k & 3) * 32) >> 4),
                             dk + (uint64_t)(((k >> 2) * Sh::kBlock + (k & 3) * 32) >> 4), id_qk, k ? 1u : 0u);
                mma_commit(&fx.s_full[s]);
                mma_commit(&fx.empty_k[st]);
                if (!both) mma_commit(&fx.empty_k[st]);  // for the slot that does not use it
            }
            __syncwarp();
        };
        auto weights = [&]() { return await(&fx.p_half[s], n_p++); };
        auto products = [&](int tile, bool first) {
            const int st = uniform(tile) % Sh::kStages, add = first ? 0 : 1;
            const uint64_t dv = desc_sw128_mn(v_at + st * Sh::kTile, Sh::kBlock);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half && !await(&fx.p_full[s], n_p - 1)) return false;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = Sh::KT / 32 * half; k < Sh::KT / 32 * (half + 1); ++k)  // 16 keys: 8 columns of weights, twice, 16 lines of V
#pragma unroll
                        for (int lo = 0; lo < 2; ++lo)
                            mma_f16_ta(tm + Sh::kO, tm + 64 * (k >> 2) + 32 * lo + 8 * (k & 3), dv + (uint64_t)(k * (16 * 128 >> 4)), id_pv, add || k || lo ? 1u : 0u);
                    if (half) {
                        mma_commit(&fx.pv_done[s]);
                        mma_commit(&fx.empty_v[st]);
                        if (!both) mma_commit(&fx.empty_v[st]);
                    }
                }
                __syncwarp();
            }
            return true;
        };
        auto drained = [&]() { return await(&fx.pv_done[s], n_p - 1); };
        for (Seg g; segment(x, grp, g); t_base += g.n) {
            both = g.rows > kTcRows;
            if (!slot_item(s, t_base, uniform(g.n), both, queries, see_k, see_v, scores, weights, products, drained)) break;
        }
        if (!ok) {  // products in flight end before their memory goes
            if (elect_one()) mma_commit(&fx.fin[s]);
            __syncwarp();
            (void)mbar_wait_limit(&fx.fin[s], 0, p.err, 1000000ull);
        }
    } else if (warp >= 4) {
        // ---------------- softmax warps ----------------
        const int s = (warp - 4) >> 2, rl = (tid - 128) & (kSlotThreads - 1);  // slot, lane within it
        const uint32_t lane_at = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t sc = tmem + 256 * s + lane_at, oc = sc + Sh::kO;
        unsigned char *qt = qs + s * Sh::kQ;
        const int words = p.head_size / 8;
        int grp = grp0, done = 0;
        bool ok = true;
        int x = x_begin;
        Seg g;
        while (ok && segment(x, grp, g)) {
            const bool both = g.rows > kTcRows;
            const int mine = both ? (s ? g.rows - kTcRows : kTcRows) : g.rows;  // pairs of the slot
            // two slots of at most 64 pairs: the second takes the other two warps' lanes, so each scheduler has one busy warp
            const int r = rl - (s && g.rows <= kTcRows / 2 ? kTcRows / 2 : 0);
            const int n = slot_tiles(g, s);
            // the pair's query, a row of the A operand: 16-byte word c of block b at word c ^ (r & 7)
            const int row0 = pl.src[g.group].row0, head0 = first_head(g.kvh, p.n_heads, p.n_kv_heads);
            const int nh = first_head(g.kvh + 1, p.n_heads, p.n_kv_heads) - head0;
            const int m = g.m0 + (both ? s * kTcRows : 0) + r, br = max(m, 0) / gq, hj = m - br * gq;
            const bool real = r >= 0 && r < mine && hj < nh;
            const uint4 *q4 = reinterpret_cast<const uint4 *>(p.q + (real ? (row0 + br) * p.q_row + (head0 + hj) * p.q_head : 0));
#pragma unroll
            for (int c = 0; c < HS / 8; ++c) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (real && c < words) {
                    v = q4[c];
                    v.x ^= ta.flip;
                    v.y ^= ta.flip;
                    v.z ^= ta.flip;
                    v.w ^= ta.flip;
                }
                *reinterpret_cast<uint4 *>(qt + (c >> 3) * Sh::kQBlock + rl * 128 + (((c & 7) ^ (rl & 7)) << 4)) = v;
            }
            fence_proxy_async_smem();
            tc_fence_before();  // acc of the segment before has been read
            if (n) mbar_arrive(&fx.q_full[s]);  // (nothing would hold this warp back until a slot without tiles had seen it)
            const bool busy = __any_sync(0xffffffffu, r >= 0 && r < mine);  // a warp without pairs only keeps the barriers going
            float base = -CUDART_INF_F, sum = 0.f;
            for (int i = 0; i < n; ++i, ++done) {
                ok = wait_or_stop(fx, &fx.s_full[s], (uint32_t)(done & 1), p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                constexpr int NC = Sh::KT / 64;
                if (busy) {
                    float v[64], mx;
                    float m4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        tmem_ld64_wait(sc + 64 * c, v);
#pragma unroll
                        for (int j = 0; j < 64; ++j) m4[j & 3] = fmaxf(m4[j & 3], v[j]);
                    }
                    mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * ta.scale_log2;
                    const bool grow = mx > base + (kLiftTc<BF> + kGrow<BF>) || (base == -CUDART_INF_F && mx > base);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float to = grow ? mx - kLiftTc<BF> : base;
                        const float f = to == -CUDART_INF_F ? 1.f : exp2f(base - to);
                        if (i) {
#pragma unroll
                            for (int c = 0; c < HS / 64; ++c) {
                                float a[64];
                                tmem_ld64_wait(oc + 64 * c, a);
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    uint32_t w[32];
#pragma unroll
                                    for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(a[32 * k + j] * f);
                                    tmem_st32(oc + 64 * c + 32 * k, w);
                                }
                            }
                        }
                        sum *= f;
                        base = to;
                    }
                    const float b0 = base == -CUDART_INF_F ? 0.f : base;
                    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        tmem_ld64_wait(sc + 64 * c, v);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t hi[16], lo[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float *at = v + 32 * h + 2 * j;
                                const float x0 = ex2(fmaf(at[0], ta.scale_log2, -b0)), x1 = ex2(fmaf(at[1], ta.scale_log2, -b0));
                                s4[j & 3] += x0 + x1;
                                hi[j] = pack16<BF>(x0, x1);
                                const float2 back = unpack16<BF>(hi[j]);
                                lo[j] = pack16<BF>(x0 - back.x, x1 - back.y);
                            }
                            tmem_st16(sc + 64 * c + 16 * h, hi);
                            tmem_st16(sc + 64 * c + 32 + 16 * h, lo);
                        }
                        if (c == 0) {
                            tmem_wait_st();
                            tc_fence_before();
                            mbar_arrive(&fx.p_half[s]);
                        }
                    }
                    sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                    tmem_wait_st();
                } else
                    mbar_arrive(&fx.p_half[s]);
                tc_fence_before();
                mbar_arrive(&fx.p_full[s]);
            }
            if (!ok) break;
            // the part: acc, complete once the slot's last second product is
            if (n) {
                ok = wait_or_stop(fx, &fx.pv_done[s], (uint32_t)((done - 1) & 1), p.err);  // (the issuing warp has seen those before)
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
            }
            if (busy) {
                const size_t at = (size_t)(g.out + (both ? s * kTcRows : s * g.rows) + r);
                if (real) reinterpret_cast<float2 *>(p.tc_ml)[at] = n ? make_float2(base, sum) : make_float2(-CUDART_INF_F, 0.f);
                if (n) {
                    float4 *dst = reinterpret_cast<float4 *>(p.tc_acc + at * p.head_size);
#pragma unroll
                    for (int c = 0; c < HS / 64; ++c) {
                        float v[64];
                        tmem_ld64_wait(oc + 64 * c, v);
                        if (real) {
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (64 * c + 4 * j < p.head_size) dst[16 * c + j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace

}  // namespace l2
