// The shared prefixes of the paged attention on the tensor cores (16-bit caches).
//
// What it computes: the parts (m, l, acc) of attn_pages.cu for the whole 128-key tiles of each
// prefix, for all (row, query head) pairs of the group and KV head at once: S = Q K^T, weights
// P = 2^(x - m), acc = P V, with pairs as the M of tcgen05.mma, keys as N of the first product and K of
// the second.
//
// How.  An item is a KV head and a run of up to 256 pairs; all (item, tile) steps are split evenly over
// one block per SM.  A block has two slots, each with 128 lanes of scores and of acc in tensor
// memory and four softmax warps: a run of more than 128 pairs gives each slot half of the pairs and the
// same tiles (K and V are read once for 256 pairs); a shorter run goes to both slots, which
// take alternate tiles, so that one slot's softmax runs beside the other's products.
//   warp 0     tiles of K and V by TMA into two rings (128-byte swizzle; a box is a page's rows
//              that fall into the tile, so pages of 8, 16, 32, 64 rows or a multiple of 128 are gathered
//              without a copy); rows past the prefix are never loaded, so nothing is masked
//   warp 1     one thread polls the barriers and issues whichever product is ready
//   warps 4-7, 8-11  slots 0 and 1: queries to shared memory, softmax, parts out
// A thread owns one pair: its row of scores is a lane of tensor memory, so max and sum need no
// exchange.  The weights go back over the scores as 16-bit values (half a step of the type, 2^-9 in bf16
// and 2^-12 in fp16 of each weight, below the output's own rounding of the sum) and are
// the A operand of the second product from there; the sums l are of the unrounded weights.  acc is
// rescaled only when a row's maximum has grown by more than 2^8 since the last time: weights
// stay below 2^8, far from either type's limits, and the result is the same.
//
// What bounds it: up to 128 pairs, reading K and V; above, the products and the exponentials in about
// equal measure.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "../../include/l2.h"
#include "attn_pages.cuh"
#include "attn_plan.cuh"
#include "l2_device.cuh"
#include "l2_pages.h"
#include "l2_tc.cuh"

namespace l2 {

namespace {

constexpr int kTcThreads = 384;
constexpr int kSlotThreads = 128;
constexpr uint32_t kBlock = kTcKeys * 128;  // 64 values of 128 rows: 16 KB
constexpr int kRing = 6;                    // most stages of a ring
constexpr float kGrow = 8.0f;               // see above

struct alignas(128) TcAttn {
    CUtensorMap kmap, vmap;
    PagesAttn p;
    int box_rows;
    float scale_log2;  // positive; the queries carry its sign
    uint32_t flip;     // 0x8000 in both halves when the scale is negative
};

template <int HS>
struct TcShape {
    static constexpr int kBlocks = HS / 64;                  // 64-value blocks of a row
    static constexpr uint32_t kTile = kBlocks * kBlock;      // a tile of K, V or queries
    static constexpr int kStagesK = HS == 64 ? 5 : 2, kStagesV = HS == 64 ? 5 : 2;
    static constexpr uint32_t kTiles = (2 + kStagesK + kStagesV) * kTile;
    static constexpr uint32_t kSmem = 1024 + 1024 + kTiles + (uint32_t)kPlanSmem;
};

struct TcFx {
    uint64_t full_k[kRing], empty_k[kRing], full_v[kRing], empty_v[kRing];
    uint64_t q_full[2], s_full[2], p_full[2], pv_done[2];
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(TcFx) <= 1024, "the fixed block must fit before the tiles");

// Whether a phase of `bar` is over, without suspending the thread.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ void tensor4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ bool stopped(const TcFx &fx) { return *reinterpret_cast<const volatile int *>(&fx.abort) != 0; }
__device__ __forceinline__ void stop(TcFx &fx) { *reinterpret_cast<volatile int *>(&fx.abort) = 1; }

// A bounded wait that also ends when another warp gave up; false: leave.
__device__ __forceinline__ bool wait_or_stop(TcFx &fx, uint64_t *bar, uint32_t parity, int *err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (stopped(fx)) return false;
        if ((i & 255u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, L2_DEV_ERR_TIMEOUT);
            stop(fx);
            return false;
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

}  // namespace

template <int HS, bool BF>
__global__ void __launch_bounds__(kTcThreads, 1) attn_pages_tc_kernel(const __grid_constant__ TcAttn ta) {
    using Sh = TcShape<HS>;
    const PagesAttn &p = ta.p;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    TcFx &fx = *reinterpret_cast<TcFx *>(smem);
    unsigned char *qs = smem + 1024;
    const uint32_t q_at = smem_u32(qs), k_at = q_at + 2 * Sh::kTile, v_at = k_at + Sh::kStagesK * Sh::kTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < Sh::kStagesK; ++i) {
            mbar_init(&fx.full_k[i], 1);
            mbar_init(&fx.empty_k[i], 1);
        }
        for (int i = 0; i < Sh::kStagesV; ++i) {
            mbar_init(&fx.full_v[i], 1);
            mbar_init(&fx.empty_v[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&fx.q_full[i], kSlotThreads);
            mbar_init(&fx.s_full[i], 1);
            mbar_init(&fx.p_full[i], kSlotThreads);
            mbar_init(&fx.pv_done[i], 1);
        }
        fence_barrier_init();
        fx.abort = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&fx.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = fx.tmem;
    // slot s: scores at columns 256 s (the weights over their first half), acc at 256 s + 128
    auto s_col = [&](int s) { return tmem + 256 * s; };
    auto o_col = [&](int s) { return tmem + 256 * s + 128; };
    if (!p.plan_in_block) pdl_wait();
    pdl_launch_dependents();  // after the wait: the warps' kernel reads the plan without one
    // planned over the queries' tiles, which only these threads' own writes reach before the first product
    const Plan pl = plan_here<kTcThreads>(p, smem + 1024 + Sh::kTiles, qs, false);
    const int T = pl.hdr[kHdrTcTiles], W = pl.hdr[kHdrTcCtas];
    const int u_begin = (int)blockIdx.x < W ? first_of(blockIdx.x, T, W) : 0;
    const int u_end = (int)blockIdx.x < W ? first_of(blockIdx.x + 1, T, W) : 0;
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    // every role walks the same segments
    auto segment = [&](int u, int &grp, Seg &g) {
        while (u >= pl.tc_t0[grp + 1]) ++grp;
        const int kt = pl.tc_kt[grp], local = u - pl.tc_t0[grp], item = local / kt;
        const int n = pl.src[grp].rows * gq, runs = tc_runs(n);
        g.group = grp;
        g.kvh = item / runs;
        const int run = item - g.kvh * runs;
        g.m0 = run * 2 * kTcRows;
        g.rows = min(2 * kTcRows, n - g.m0);
        g.k0 = local - item * kt;
        g.n = min(kt - g.k0, u_end - u);
        g.out = pl.tc_r0[grp] + g.kvh * tc_head_rows(n) + g.m0 + 2 * kTcRows * (int)blockIdx.x;
    };
    // tiles slot s works on, and the tile of its i-th
    auto slot_tiles = [&](const Seg &g, int s) { return g.rows > kTcRows ? g.n : (g.n + 1 - s) >> 1; };
    auto slot_tile = [&](const Seg &g, int s, int i) { return g.rows > kTcRows ? i : 2 * i + s; };
    int grp0 = 0;
    if (u_begin < u_end) grp0 = warp_find(pl.tc_t0, 1, p.G + 1, u_begin);

    if (warp == 0) {
        // ---------------- copies: lane j issues box j of a tile ----------------
        int t = 0, grp = grp0;
        const int boxes = kTcKeys / ta.box_rows;
        bool ok = true;
        for (int u = u_begin; u < u_end && ok;) {
            Seg g;
            segment(u, grp, g);
            u += g.n;
            const int r0 = pl.src[g.group].row0;
            const int *table = p.table + (size_t)(p.seqs ? p.seqs[r0] : r0) * p.max_pages;
            auto lookup = [&](int tile) {
                const int pos = (g.k0 + tile) * kTcKeys + lane * ta.box_rows;
                return lane < boxes && tile < g.n ? table[page_of(p, pos)] : 0;
            };
            // one tile of K or V; its page ids were loaded a step before
            auto copy = [&](int kv, int tile, int tt, int page) {
                const int ns = kv ? Sh::kStagesV : Sh::kStagesK, st = tt % ns;
                uint64_t *full = kv ? &fx.full_v[st] : &fx.full_k[st], *empty = kv ? &fx.empty_v[st] : &fx.empty_k[st];
                if (tt >= ns) ok = wait_or_stop(fx, empty, (uint32_t)((tt / ns - 1) & 1), p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                if (lane == 0) mbar_arrive_expect_tx(full, Sh::kTile);
                __syncwarp();
                if (lane < boxes) {
                    const int pos = (g.k0 + tile) * kTcKeys + lane * ta.box_rows, row = pos - page_of(p, pos) * p.page_size;
                    const int cp = page >= 0 && page < p.n_pages ? page : p.n_pages;  // out of range: TMA fills zeros
                    if (cp == p.n_pages) atomicOr(p.err, L2_DEV_ERR_BOUNDS);
                    const uint32_t dst = (kv ? v_at : k_at) + st * Sh::kTile + lane * ta.box_rows * 128;
#pragma unroll
                    for (int b = 0; b < Sh::kBlocks; ++b) tensor4d(dst + b * kBlock, kv ? &ta.vmap : &ta.kmap, 64 * b, row, g.kvh, cp, full);
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
        // copies in flight land before the block's memory goes (all have, when the others finished)
        if (!ok) {
            for (int st = 0; st < Sh::kStagesK; ++st)
                for (int ph = 0; ph < 2; ++ph) (void)mbar_wait_limit(&fx.full_k[st], ph, p.err, 1000000ull);
            for (int st = 0; st < Sh::kStagesV; ++st)
                for (int ph = 0; ph < 2; ++ph) (void)mbar_wait_limit(&fx.full_v[st], ph, p.err, 1000000ull);
        }
    } else if (warp == 1) {
        // ---------------- products: one thread, whichever is ready ----------------
        if (lane == 0) {
            int grp = grp0, t_base = 0;
            int nqk[2] = {0, 0}, npv[2] = {0, 0}, nseg = 0;  // products issued per slot, segments begun
            const uint32_t id_qk = idesc_f16(BF, kTcRows, kTcKeys, false), id_pv = idesc_f16(BF, kTcRows, HS, true);
            bool ok = true;
            for (int u = u_begin; u < u_end && ok; ++nseg) {
                Seg g;
                segment(u, grp, g);
                u += g.n;
                const bool both = g.rows > kTcRows;
                int qk[2] = {0, 0}, pv[2] = {0, 0};
                const int cnt[2] = {slot_tiles(g, 0), slot_tiles(g, 1)};
                bool q_in[2] = {false, false};
                uint32_t idle = 0;
                uint64_t t_idle = 0;
                while (pv[0] < cnt[0] || pv[1] < cnt[1]) {
                    bool moved = false;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        // the weights of the slot's last scores are in: the second product
                        if (pv[s] < qk[s]) {
                            const int t = t_base + slot_tile(g, s, pv[s]), st = t % Sh::kStagesV;
                            if (mbar_test(&fx.p_full[s], (uint32_t)(npv[s] & 1)) &&
                                mbar_test(&fx.full_v[st], (uint32_t)((t / Sh::kStagesV) & 1))) {
                                tc_fence_after();
                                const uint64_t dv = desc_sw128_mn(v_at + st * Sh::kTile, kBlock);
#pragma unroll
                                for (int k = 0; k < kTcKeys / 16; ++k)  // 16 keys: 8 columns of weights, 16 lines of V
                                    mma_f16_ta(o_col(s), s_col(s) + 8 * k, dv + (uint64_t)(k * (16 * 128 >> 4)), id_pv, pv[s] || k ? 1u : 0u);
                                ++pv[s];
                                ++npv[s];
                                mma_commit(&fx.pv_done[s]);
                                if (!both || pv[s ^ 1] >= pv[s]) mma_commit(&fx.empty_v[st]);
                                moved = true;
                            }
                        }
                        // the slot's scores are free (its last second product is over): the first product of its next tile
                        if (qk[s] < cnt[s] && pv[s] == qk[s]) {
                            const int t = t_base + slot_tile(g, s, qk[s]), st = t % Sh::kStagesK;
                            if (!q_in[s]) q_in[s] = mbar_test(&fx.q_full[s], (uint32_t)(nseg & 1));
                            if (q_in[s] && (npv[s] == 0 || mbar_test(&fx.pv_done[s], (uint32_t)((npv[s] - 1) & 1))) &&
                                mbar_test(&fx.full_k[st], (uint32_t)((t / Sh::kStagesK) & 1))) {
                                tc_fence_after();
                                const uint64_t dq = desc_sw128(q_at + s * Sh::kTile), dk = desc_sw128(k_at + st * Sh::kTile);
#pragma unroll
                                for (int k = 0; k < HS / 16; ++k) {  // 32 bytes a step, blocks of 4 steps
                                    const uint64_t off = (uint64_t)(((k >> 2) * kBlock + (k & 3) * 32) >> 4);
                                    mma_bf16(s_col(s), dq + off, dk + off, id_qk, k ? 1u : 0u);
                                }
                                ++qk[s];
                                ++nqk[s];
                                mma_commit(&fx.s_full[s]);
                                if (!both || qk[s ^ 1] >= qk[s]) mma_commit(&fx.empty_k[st]);
                                moved = true;
                            }
                        }
                    }
                    if (moved) {
                        idle = 0;
                    } else if ((++idle & 255u) == 0) {
                        const uint64_t now = globaltimer_ns();
                        if (idle == 256u) t_idle = now;
                        if (stopped(fx) || now - t_idle > kWaitLimitNs) {
                            if (!stopped(fx)) atomicOr(p.err, L2_DEV_ERR_TIMEOUT);
                            stop(fx);
                            ok = false;
                            break;
                        }
                    }
                }
                t_base += g.n;
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------- softmax warps ----------------
        const int s = (warp - 4) >> 2, rl = (tid - 128) & (kSlotThreads - 1);  // slot, lane within it
        const uint32_t lane_at = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t sc = s_col(s) + lane_at, oc = o_col(s) + lane_at;
        unsigned char *qt = qs + s * Sh::kTile;
        const int words = p.head_size / 8;
        int grp = grp0, done = 0;
        bool ok = true;
        for (int u = u_begin; u < u_end && ok;) {
            Seg g;
            segment(u, grp, g);
            u += g.n;
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
                *reinterpret_cast<uint4 *>(qt + (c >> 3) * kBlock + rl * 128 + (((c & 7) ^ (rl & 7)) << 4)) = v;
            }
            fence_proxy_async_smem();
            tc_fence_before();  // acc of the segment before has been read
            mbar_arrive(&fx.q_full[s]);
            const bool busy = __any_sync(0xffffffffu, r >= 0 && r < mine);  // a warp without pairs only keeps the barriers going
            float base = -CUDART_INF_F, sum = 0.f;
            for (int i = 0; i < n; ++i, ++done) {
                ok = wait_or_stop(fx, &fx.s_full[s], (uint32_t)(done & 1), p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (busy) {
                    float v[64], m4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tmem_ld64_wait(sc + 64 * c, v);
#pragma unroll
                        for (int j = 0; j < 64; ++j) m4[j & 3] = fmaxf(m4[j & 3], v[j]);
                    }
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * ta.scale_log2;
                    const bool grow = mx > base + kGrow || (base == -CUDART_INF_F && mx > base);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float to = grow ? mx : base;
                        const float f = to == -CUDART_INF_F ? 1.f : exp2f(base - to);
                        if (i) {
#pragma unroll
                            for (int c = 0; c < HS / 64; ++c) {
                                tmem_ld64_wait(oc + 64 * c, v);
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    uint32_t w[32];
#pragma unroll
                                    for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[32 * k + j] * f);
                                    tmem_st32(oc + 64 * c + 32 * k, w);
                                }
                            }
                        }
                        sum *= f;
                        base = to;
                    }
                    const float b0 = base == -CUDART_INF_F ? 0.f : base;
                    // weights of scores 64 c .. go over columns 32 c .., read by then
                    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tmem_ld64_wait(sc + 64 * c, v);
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float x = ex2(fmaf(v[2 * j], ta.scale_log2, -b0)), y = ex2(fmaf(v[2 * j + 1], ta.scale_log2, -b0));
                            s4[j & 3] += x + y;
                            w[j] = pack16<BF>(x, y);
                        }
                        tmem_st32(sc + 32 * c, w);
                    }
                    sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(&fx.p_full[s]);
            }
            if (!ok) break;
            // the part: acc, complete once the slot's last second product is
            if (n) {
                ok = wait_or_stop(fx, &fx.pv_done[s], (uint32_t)((done - 1) & 1), p.err);
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

namespace {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Rows of a page that one box takes.
int box_rows(int page_size) { return page_size < kTcKeys ? page_size : kTcKeys; }

// Pages as a tensor (value, row, KV head, page), in boxes of 64 values by `rows` rows.
bool encode_pages(CUtensorMap *m, const char *base, const PagesAttn &p, int rows) {
    EncodeFn fn = reinterpret_cast<EncodeFn>(tensor_map_encoder());
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)p.head_size, (cuuint64_t)p.page_size, (cuuint64_t)p.n_kv_heads, (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.row_stride, (cuuint64_t)p.head_stride, (cuuint64_t)p.page_stride};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, p.dtype == L2_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<char *>(base),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HS, bool BF>
cudaError_t launch_tc(const TcAttn &ta, cudaLaunchConfig_t cfg) {
    auto fn = attn_pages_tc_kernel<HS, BF>;
    static DeviceOnce once;
    cudaError_t e = once.smem(reinterpret_cast<const void *>(fn), (int)TcShape<HS>::kSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(ta.p.num_sms);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = TcShape<HS>::kSmem;
    return cudaLaunchKernelEx(&cfg, fn, ta);
}

}  // namespace

// A box must start at a page row and cover whole groups of 8 lines of the swizzle: pages of 8, 16, 32, 64 rows or
// a multiple of 128; a tensor's strides are below 2^40 bytes.
bool attn_pages_tc_supported(const PagesAttn &p) {
    if (p.dtype != L2_BF16 && p.dtype != L2_F16) return false;
    const bool whole = p.page_size % kTcKeys == 0, part = p.page_size >= 8 && kTcKeys % p.page_size == 0;
    const long long lim = 1ll << 40;
    return (whole || part) && p.row_stride < lim && p.head_stride < lim && p.page_stride < lim && tensor_map_encoder();
}

cudaError_t launch_attn_pages_tc(const PagesAttn &p, cudaLaunchConfig_t cfg) {
    TcAttn ta{};
    ta.p = p;
    ta.box_rows = box_rows(p.page_size);
    ta.scale_log2 = p.scale_log2 < 0.f ? -p.scale_log2 : p.scale_log2;
    ta.flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    if (!encode_pages(&ta.kmap, p.k, p, ta.box_rows) || !encode_pages(&ta.vmap, p.v, p, ta.box_rows)) return cudaErrorInvalidValue;
    if (p.head_size <= 64) return p.dtype == L2_BF16 ? launch_tc<64, true>(ta, cfg) : launch_tc<64, false>(ta, cfg);
    return p.dtype == L2_BF16 ? launch_tc<128, true>(ta, cfg) : launch_tc<128, false>(ta, cfg);
}

}  // namespace l2
