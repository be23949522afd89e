// The shared prefixes of the paged attention over fp32 caches on the tensor cores: one role of the blocks of
// attn_pages_f32.cu.
//
// What it computes: the parts (m, l, acc) of attn_pages.cu for the whole 64-key tiles of each prefix, for
// all (row, query head) pairs of the group and KV head at once, to fp32's own accuracy.
//
// How.  Every operand (q, K, the weights 2^(x - m), V) is cut into three bf16 values that add up to it exactly: the top 8
// bits as they stand (so a finite value stays finite), 8 more rounded, and the rest.  Of the nine products of two such sums
// the six largest are taken; what is left out is 2^-24 of a product, of either sign.  The tensor core cuts the sums it adds
// into, so the small products go first and the largest last: an accumulator meets a score's full size
// in HS / 16 additions, and a tile's sums leave tensor memory after every tile and are added in fp32 registers.  (tf32 halves
// would take half the products at half the rate, and V^T in shared memory, since tf32 operands are K-major.)
//   warp 0     the products: S = Q K^T (Q in tensor memory), then P V (P in tensor memory)
//   warps 1-3  K and V: a tile's rows are copied through the page table (a bulk copy for the rows of a page, so pages may
//              have any size), cut, and stored as three 128-byte-swizzled operands
//   warps 4-7, 8-11  two warpgroups over the same 128 pairs: a thread owns a pair, reads all its scores (the max
//              needs no exchange) and makes the weights of half of the keys and the sums of half of the head
// Tensor memory: Q 3 HS / 2 columns, S 64, P 96, the tile's sums HS; head sizes up to 64 leave room for a second tile of
// scores, which is then issued two tiles ahead, and otherwise as soon as S has been read.
//
// What bounds it: the warps that cut K and V.  A tile takes 2.4 us at head size 64 and 3.4 at 128, whatever its pairs, and as long
// with one product of the six; an SM's walkers take 2.5 and 6 for 32 pairs, 10 and 24 for 128.  (Copies by cp.async from every
// cutting warp: 2.5 and 3.4; plain loads: 6.4 and 13.)
#pragma once
#include "attn_pages_tc.cuh"

namespace l2 {

namespace {

template <int HS>
struct Tc32Shape {
    static constexpr int KT = tc_keys(true);
    static constexpr int kBlocks = HS / 64;                             // 64-value blocks of a row
    static constexpr uint32_t kBlock = KT * 128, kSplit = kBlocks * kBlock, kTile = 3 * kSplit;
    static constexpr int kStages = HS == 64 ? 2 : 1;                    // tiles of K, and of V, as operands
    static constexpr uint32_t kRaw = KT * HS * 4;                       // a tile of K or V as it is read (of HS at most)
    static constexpr int kRawStages = HS == 64 ? 6 : 3;
    static constexpr uint32_t kSmem = 1024 + 1024 + 2 * kStages * kTile + kRawStages * kRaw;  // alignment, barriers, tiles
    static constexpr int kAhead = HS == 64 ? 2 : 1;                     // tiles of scores
    static constexpr int kQ = 0, kS = 3 * HS / 2, kP = kS + kAhead * KT, kO = kP + 3 * KT / 2;
    static_assert(kO + HS <= 512, "tensor memory has 512 columns");
};

struct Tc32Fx {
    uint64_t full_k[2], empty_k[2], full_v[2], empty_v[2];
    uint64_t raw_full[6], raw_empty[6], s_full[2], q_full, p_full, pv_done, l_full, fin;
    uint64_t seen[4];    // the two warps of a lane quarter have read the scores that they are about to write
    uint32_t tmem;
    int abort;
    unsigned bad[6][2];  // rows of a tile whose page is out of range
    float l[kTcRows];    // the second warpgroup's sums
};
static_assert(sizeof(Tc32Fx) <= 1024, "the fixed block must fit before the tiles");

constexpr int kCutWarps = 3;

// x and y as three pairs of bf16 values.
__device__ __forceinline__ void cut3(float x, float y, uint32_t *w) {
    const uint32_t xb = __float_as_uint(x), yb = __float_as_uint(y);
    w[0] = __byte_perm(xb, yb, 0x7632);
    x -= __uint_as_float(xb & 0xffff0000u);
    y -= __uint_as_float(yb & 0xffff0000u);
    const __nv_bfloat162 m = __floats2bfloat162_rn(x, y);
    w[1] = *reinterpret_cast<const uint32_t *>(&m);
    x -= __uint_as_float(w[1] << 16);
    y -= __uint_as_float(w[1] & 0xffff0000u);
    w[2] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);  // at most 8 bits are left
}

__device__ __forceinline__ void tmem_st1(uint32_t addr, uint32_t v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 32 columns of the warp's lanes, complete when it returns.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t addr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}

// One block's work, all of its threads.  smem: kSmem bytes; pl: the plan; bid: the block among those of the role.
template <int HS>
__device__ __forceinline__ void tc32_role(const PagesAttn &p, const Plan &pl, unsigned char *smem_raw, int bid) {
    using Sh = Tc32Shape<HS>;
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Tc32Fx &fx = *reinterpret_cast<Tc32Fx *>(smem);
    const uint32_t k_at = smem_u32(smem + 1024), v_at = k_at + Sh::kStages * Sh::kTile;
    unsigned char *raw_mem = smem + 1024 + 2 * Sh::kStages * Sh::kTile;
    const uint32_t raw_at = smem_u32(raw_mem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            mbar_init(&fx.full_k[i], kCutWarps);
            mbar_init(&fx.empty_k[i], 1);
            mbar_init(&fx.full_v[i], kCutWarps);
            mbar_init(&fx.empty_v[i], 1);
        }
        for (int i = 0; i < Sh::kRawStages; ++i) {
            mbar_init(&fx.raw_full[i], 1);
            mbar_init(&fx.raw_empty[i], kCutWarps);
        }
        mbar_init(&fx.q_full, 2 * kSlotThreads);
        mbar_init(&fx.s_full[0], 1);
        mbar_init(&fx.s_full[1], 1);
        mbar_init(&fx.p_full, 2 * kSlotThreads);
        mbar_init(&fx.pv_done, 1);
        mbar_init(&fx.l_full, kSlotThreads);
        mbar_init(&fx.fin, 1);
        for (int i = 0; i < 4; ++i) mbar_init(&fx.seen[i], 2);
        fence_barrier_init();
        fx.abort = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&fx.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_proxy_async_smem();  // the plan was built over the tiles' memory
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = fx.tmem;
    const int x_begin = bid * pl.hdr[kHdrTcPer], x_end = min(x_begin + pl.hdr[kHdrTcPer], pl.hdr[kHdrTcCost]);
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads), words = p.head_size / 4;
    int x = x_begin, grp = x_begin < x_end ? warp_find(pl.tc_t0, 1, p.G + 1, x_begin) : 0;
    auto segment = [&](Seg &g) { return tc_segment<true>(p, pl, gq, bid, x_end, x, grp, g); };
    bool ok = true;
    auto await = [&](uint64_t *bar, int parity) {
        ok = __all_sync(0xffffffffu, wait_or_stop(fx, bar, (uint32_t)parity & 1u, p.err));
        return ok;
    };
    // byte offset of a key's row of a sequence, -1 where the table is bad
    auto row_of = [&](const int *table, int kvh, int key, int page) {
        return page >= 0 && page < p.n_pages
                   ? kvh * p.head_stride + page * p.page_stride + (key - page_of(p, key) * p.page_size) * p.row_stride
                   : -1ll;
    };
    Seg g;

    if (warp == 0) {
        // ---------------- products ----------------
        auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
        const uint32_t tm = (uint32_t)uniform((int)tmem);
        const uint32_t id_qk = idesc_f16(true, kTcRows, Sh::KT, false), id_pv = idesc_f16(true, kTcRows, HS, true);
        // parts of A and B of product o, 0 the largest: the smallest products first.  (Loops over o stay loops:
        // unrolled they were six times the code and no faster.)
        auto part_a = [](int o) { return 0x001102 >> 4 * o & 3; };
        auto part_b = [](int o) { return 0x010120 >> 4 * o & 3; };
        int t0 = 0, n_p = 0, nseg = 0;  // tiles before the item, second products, items begun
        for (; ok && segment(g); ++nseg) {
            const int n = uniform(g.n);
            auto scores = [&](int i) {
                const int t = uniform(t0 + i), st = t % Sh::kStages;
                if (!await(&fx.full_k[st], t / Sh::kStages)) return;
                tc_fence_after();
                const uint64_t dk = desc_sw128(k_at + st * Sh::kTile);
                if (elect_one()) {
#pragma unroll 1
                    for (int o = 0; o < 6; ++o)
#pragma unroll
                        for (int k = 0; k < HS / 16; ++k)
                            mma_f16_ta(tm + Sh::kS + (t % Sh::kAhead) * Sh::KT, tm + Sh::kQ + part_a(o) * (HS / 2) + 8 * k,
                                       dk + (uint64_t)((part_b(o) * Sh::kSplit + (k >> 2) * Sh::kBlock + (k & 3) * 32) >> 4), id_qk, o || k ? 1u : 0u);
                    mma_commit(&fx.s_full[t % Sh::kAhead]);
                    mma_commit(&fx.empty_k[st]);
                }
                __syncwarp();
            };
            if (!await(&fx.q_full, nseg)) break;
            scores(0);
            if (ok && Sh::kAhead == 2 && n > 1) scores(1);
            for (int i = 0; i < n && ok; ++i) {
                const int t = uniform(t0 + i), st = t % Sh::kStages;
                if (!await(&fx.p_full, n_p)) break;  // the weights are there, and the scores read
                ++n_p;
                if (Sh::kAhead == 1 && i + 1 < n) scores(i + 1);
                if (!ok || !await(&fx.full_v[st], t / Sh::kStages)) break;
                tc_fence_after();
                const uint64_t dv = desc_sw128_mn(v_at + st * Sh::kTile, Sh::kBlock);
                if (elect_one()) {
#pragma unroll 1
                    for (int o = 0; o < 6; ++o)
#pragma unroll
                        for (int k = 0; k < Sh::KT / 16; ++k)
                            mma_f16_ta(tm + Sh::kO, tm + Sh::kP + part_a(o) * (Sh::KT / 2) + 8 * k,
                                       dv + (uint64_t)((part_b(o) * Sh::kSplit + k * 16 * 128) >> 4), id_pv, o || k ? 1u : 0u);
                    mma_commit(&fx.pv_done);
                    mma_commit(&fx.empty_v[st]);
                }
                __syncwarp();
                if (Sh::kAhead == 2 && i + 2 < n) scores(i + 2);
            }
            t0 += g.n;
        }
        if (!ok) {  // products in flight end before their memory goes
            if (elect_one()) mma_commit(&fx.fin);
            __syncwarp();
            (void)mbar_wait_limit(&fx.fin, 0, p.err, 1000000ull);
        }
    } else if (warp <= kCutWarps) {
        // ---------------- K and V ----------------
        // The warps copy in turn, and all three cut: one instruction reads RP rows, and a warp takes every third such group.
        constexpr int LR = HS / 4, RP = 32 / LR, kGroups = Sh::KT / RP, kMine = (kGroups + kCutWarps - 1) / kCutWarps, kRaws = Sh::kRawStages, kDist = HS == 64 ? kRaws - 1 : kRaws;
        const int rr = lane / LR, c = lane % LR, pitch = words * 16;
        const uint32_t raw = raw_at + rr * pitch + c * 16, col = (uint32_t)((c >> 4) * Sh::kBlock + (c & 1) * 8);
        const int word = (c & 15) >> 1;
        const bool run_on = p.row_stride == pitch;  // rows of a page lie behind one another
        int t0 = 0, copied = 0, cut = 0;            // tiles before the item, operations (tiles of K or V) copied and cut
        while (ok && segment(g)) {
            const int *table = p.table + (size_t)pl.src[g.group].seq * p.max_pages;
            const int n_ops = 2 * g.n;  // K 0, K 1, V 0, K 2, V 1, .., V n - 1
            auto is_v = [&](int op) { return op && (!(op & 1) || op == n_ops - 1); };
            auto tile = [&](int op) { return op == 0 ? 0 : op & 1 ? min((op + 1) >> 1, g.n - 1) : (op >> 1) - 1; };
            static_assert(kRaws % kCutWarps == 0, "a stage is always copied to by the same warp, which has seen all of its releases");
            int pages[2];  // of keys lane and lane + 32 of the tile this warp copies next
            auto look = [&](int op) {
                if (op >= n_ops) return;
                const int key = (g.k0 + tile(op)) * Sh::KT + lane;
                pages[0] = table[page_of(p, key)];
                pages[1] = table[page_of(p, key + 32)];
            };
            // a copy for each stretch of rows that lie in one page; rows of a bad page are marked
            auto copy = [&](int op) {
                if (op >= n_ops) return;
                const int u = copied++, st = u % kRaws, key = (g.k0 + tile(op)) * Sh::KT + lane;
                if (u % kCutWarps != warp - 1 || (u >= kRaws && !await(&fx.raw_empty[st], u / kRaws - 1))) return;
                long long off[2];
                unsigned bad[2];
                int n[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = key + 32 * h, in_page = k - page_of(p, k) * p.page_size;
                    off[h] = row_of(table, g.kvh, k, pages[h]);
                    bad[h] = __ballot_sync(0xffffffffu, off[h] < 0);
                    if (off[h] < 0) atomicOr(p.err, L2_DEV_ERR_BOUNDS);
                    const bool first = !run_on || in_page == 0 || (lane == 0 && h == 0);
                    n[h] = off[h] < 0 || !first ? 0 : run_on ? min(p.page_size - in_page, Sh::KT - lane - 32 * h) : 1;
                }
                look(op + kCutWarps);
                if (lane == 0) {
                    fx.bad[st][0] = bad[0];
                    fx.bad[st][1] = bad[1];
                    mbar_arrive_expect_tx(&fx.raw_full[st], (Sh::KT - __popc(bad[0]) - __popc(bad[1])) * pitch);
                }
                __syncwarp();
                const char *base = is_v(op) ? p.v : p.k;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (n[h]) bulk_g2s_nohint(raw_mem + st * Sh::kRaw + (lane + 32 * h) * pitch, base + off[h], n[h] * pitch, &fx.raw_full[st]);
                __syncwarp();
            };
            look((warp - 1 + kCutWarps - copied % kCutWarps) % kCutWarps);
#pragma unroll 1
            for (int op = 1 - kDist; op < n_ops && ok; ++op) {
                copy(op + kDist - 1);
                if (op < 0) continue;
                const int t = t0 + tile(op), st = t % Sh::kStages, rs = cut % kRaws;
                const bool v = is_v(op);
                if (!ok || (t >= Sh::kStages && !await(v ? &fx.empty_v[st] : &fx.empty_k[st], t / Sh::kStages - 1))) break;
                if (!await(&fx.raw_full[rs], cut / kRaws)) break;
                ++cut;
                const unsigned bad[2] = {fx.bad[rs][0], fx.bad[rs][1]};
                const uint32_t from = raw + rs * Sh::kRaw, to = (v ? v_at : k_at) + st * Sh::kTile + col;
                constexpr int kAtOnce = 11;  // words in flight a lane
#pragma unroll
                for (int j0 = 0; j0 < kMine; j0 += kAtOnce) {
                    float4 x[kAtOnce];
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j) {
                        const int at = min(warp - 1 + kCutWarps * (j0 + j), kGroups - 1);
                        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (c < words)
                            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[j].x), "=f"(x[j].y), "=f"(x[j].z), "=f"(x[j].w) : "r"(from + at * RP * pitch));
                    }
                    if (bad[0] | bad[1]) {
#pragma unroll
                        for (int j = 0; j < kAtOnce; ++j) {
                            const int row = min(warp - 1 + kCutWarps * (j0 + j), kGroups - 1) * RP + rr;
                            if ((row & 32 ? bad[1] : bad[0]) >> (row & 31) & 1) x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    }
                    uint32_t lo[kAtOnce][3], hi[kAtOnce][3];
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j) {
                        cut3(x[j].x, x[j].y, lo[j]);
                        cut3(x[j].z, x[j].w, hi[j]);
                    }
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j) {
                        const int at = warp - 1 + kCutWarps * (j0 + j), row = at * RP + rr;
                        if (at >= kGroups) continue;
                        const uint32_t a = to + row * 128 + ((word ^ (row & 7)) << 4);
#pragma unroll
                        for (int s = 0; s < 3; ++s)
                            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a + s * Sh::kSplit), "r"(lo[j][s]), "r"(hi[j][s]) : "memory");
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&fx.raw_empty[rs]);
                    mbar_arrive(v ? &fx.full_v[st] : &fx.full_k[st]);
                }
            }
            t0 += g.n;
        }
        // the last stages' releases land before the block's memory goes; copies in flight do where something gave up
        for (int t = max(0, t0 - Sh::kStages); t < t0 && ok; ++t) {
            const int st = t % Sh::kStages;
            if (await(&fx.empty_k[st], t / Sh::kStages)) await(&fx.empty_v[st], t / Sh::kStages);
        }
        if (!ok) {
            for (int st = 0; st < kRaws; ++st)
                for (int ph = 0; ph < 2; ++ph) (void)mbar_wait_limit(&fx.raw_full[st], ph, p.err, 1000000ull);
        }
    } else {
        // ---------------- weights and sums ----------------
        const int w = (warp - walk_first(true)) >> 2, r = (tid - 32 * walk_first(true)) & (kSlotThreads - 1);  // warpgroup, pair
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        constexpr int HD = HS / 2;  // dimensions of the sums a warpgroup keeps
        // the queries carry the scale's sign, so the largest score is the largest product
        const float scale = fabsf(p.scale_log2), sign = p.scale_log2 < 0.f ? -1.f : 1.f;
        int done = 0, ended = 0, nseg = 0, odd = 0;
        for (; ok && segment(g); ++nseg) {
            const int row0 = pl.src[g.group].row0, head0 = first_head(g.kvh, p.n_heads, p.n_kv_heads);
            const int nh = first_head(g.kvh + 1, p.n_heads, p.n_kv_heads) - head0;
            const int m = g.m0 + r, br = m / gq, hj = m - br * gq;
            const bool real = r < g.rows && hj < nh;
            const float4 *q4 = reinterpret_cast<const float4 *>(p.q + (real ? (row0 + br) * p.q_row + (head0 + hj) * p.q_head : 0));
            if (w < Sh::kBlocks) {  // 64 values of the query
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t cut[3][16];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int at = 16 * w + 8 * h + c;
                        const float4 v = real && at < words ? q4[at] : make_float4(0.f, 0.f, 0.f, 0.f);
                        uint32_t lo[3], hi[3];
                        cut3(v.x * sign, v.y * sign, lo);
                        cut3(v.z * sign, v.w * sign, hi);
#pragma unroll
                        for (int s = 0; s < 3; ++s) {
                            cut[s][2 * c] = lo[s];
                            cut[s][2 * c + 1] = hi[s];
                        }
                    }
#pragma unroll
                    for (int s = 0; s < 3; ++s) tmem_st16(tl + Sh::kQ + s * (HS / 2) + 32 * w + 16 * h, cut[s]);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            mbar_arrive(&fx.q_full);
            const bool busy = __any_sync(0xffffffffu, r < g.rows);  // a warp without pairs only keeps the barriers going
            float base = -CUDART_INF_F, sum = 0.f, acc[HD];
#pragma unroll
            for (int j = 0; j < HD; ++j) acc[j] = 0.f;
            auto add_sums = [&]() {
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    float v[32];
                    tmem_ld32_wait(tl + Sh::kO + w * HD + 32 * c, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[32 * c + j] += v[j];
                }
            };
            for (int i = 0; i < g.n; ++i, ++done) {
                if (!await(&fx.s_full[done % Sh::kAhead], done / Sh::kAhead)) break;
                tc_fence_after();
                const uint32_t sc = tl + Sh::kS + (done % Sh::kAhead) * Sh::KT;
                float mx = -CUDART_INF_F;
                if (busy) {
                    float m4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int c = 0; c < Sh::KT / 32; ++c) {
                        float v[32];
                        tmem_ld32_wait(sc + 32 * c, v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) m4[j & 3] = max_nan(m4[j & 3], v[j]);
                    }
                    mx = max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3]));
                    // the parts of an infinity make NaN of a score that may be infinite: such tiles are summed again as they are
                    // (by both warps of the lanes, which read the same scores, so both come here; each then writes its own keys')
                    if (__any_sync(0xffffffffu, mx != mx && real)) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&fx.seen[warp & 3]);
                        if (!await(&fx.seen[warp & 3], odd++)) break;
                        tc_fence_after();
                        mx = -CUDART_INF_F;
                        const int *table = p.table + (size_t)pl.src[g.group].seq * p.max_pages;
#pragma unroll 1
                        for (int j = 0; j < Sh::KT; ++j) {
                            const int key = (g.k0 + i) * Sh::KT + j;
                            const long long o = row_of(table, g.kvh, key, table[page_of(p, key)]);
                            const float4 *k4 = reinterpret_cast<const float4 *>(p.k + o);
                            float d = 0.f;
                            if (real && o >= 0)
#pragma unroll 1
                                for (int c = 0; c < words; ++c) {
                                    const float4 a = q4[c], b = k4[c];
                                    d = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, d))));
                                }
                            d *= sign;
                            if (j / (Sh::KT / 2) == w) tmem_st1(sc + j, __float_as_uint(d));
                            mx = fmaxf(mx, d);
                        }
                        tmem_wait_st();
                    }
                    mx *= scale;
                }
                uint32_t cut[3][16];
                float f = 1.f;
                // the weights of this warpgroup's keys
                auto weights = [&]() {
                    if (!busy) return;
                    const float mn = fmaxf(base, mx), b0 = mn == -CUDART_INF_F ? 0.f : mn;
                    f = exp2f(base - b0);
                    base = mn;
                    float v[32], s4[4] = {0.f, 0.f, 0.f, 0.f};
                    tmem_ld32_wait(sc + 32 * w, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float x0 = ex2(fmaf(v[2 * j], scale, -b0)), x1 = ex2(fmaf(v[2 * j + 1], scale, -b0));
                        s4[j & 3] += x0 + x1;
                        uint32_t x3[3];
                        cut3(x0, x1, x3);
                        cut[0][j] = x3[0];
                        cut[1][j] = x3[1];
                        cut[2][j] = x3[2];
                    }
                    sum = sum * f + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
                };
                // where registers hold them and the sums, they are made before the wait for their columns
                if (Sh::kAhead == 2) weights();
                if (i) {  // the product before: its sums are complete and its weights read
                    if (!await(&fx.pv_done, ended++)) break;
                    tc_fence_after();
                    if (busy) add_sums();
                }
                if (Sh::kAhead == 1) weights();
                if (busy) {
#pragma unroll
                    for (int s = 0; s < 3; ++s) tmem_st16(tl + Sh::kP + s * (Sh::KT / 2) + 16 * w, cut[s]);
                    if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
                        for (int j = 0; j < HD; ++j) acc[j] *= f;
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(&fx.p_full);
            }
            if (w == 1) {  // read again only in the next item, whose scores wait for the first warpgroup's queries
                fx.l[r] = sum;
                mbar_arrive(&fx.l_full);
            }
            if (!ok || !await(&fx.pv_done, ended++) || (w == 0 && !await(&fx.l_full, nseg))) break;
            tc_fence_after();
            if (busy) {
                add_sums();
                if (real) {
                    const size_t at = (size_t)(g.out + r);
                    if (w == 0) reinterpret_cast<float2 *>(p.tc_ml)[at] = make_float2(base, sum + fx.l[r]);
                    float4 *dst = reinterpret_cast<float4 *>(p.tc_acc + at * p.head_size);
#pragma unroll
                    for (int j = 0; j < HD / 4; ++j)
                        if (w * HD + 4 * j < p.head_size) dst[w * (HD / 4) + j] = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
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
