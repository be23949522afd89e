// Decode attention of a batch over a paged cache whose sequences share prefixes.
//
// What it computes.  For row b (the newest token of sequence s_b, lens[s_b] = n rows cached),
// query head h and its KV head g(h) = floor(h * n_kv_heads / n_heads):
//     x_t = scale * q_bh . K[t, g(h)],  o_bh = sum_t softmax(x)_t V[t, g(h)],  t = 0 .. n - 1.
// The batch comes in groups; the first P_g positions of a group (the group's prefix length, at
// most the shortest member's length) are read through its first sequence's table, once for all
// its rows, and the rest through each sequence's own.
//
// How.  A softmax over keys splits over any partition of them: each part keeps (m, l, acc) = (max
// of x, sum of 2^(x - m), sum of 2^(x - m) V) in base 2, and parts merge by rescaling to the common max.
// "Sources" are the groups' prefixes and then the sequences' own rows; a source has items, one
// per KV head and tile of 16 (row, head) pairs, and an item's keys are cut into tiles.  All tiles,
// numbered source by source, are split evenly over the warps of the grid; a warp walks its range
// and writes one part per item it meets (item number + warp number is a distinct slot, because
// each step from part to part raises one of the two).  A second kernel merges each row's
// parts in key order, so results do not depend on timing.
//
// What bounds it.  16 rows against a tile give 16 products per word read, so the reading of K and V bounds
// the kernel until a prefix serves many tiles of rows.  Each warp keeps its own ring of tiles
// (cp.async, 16-byte words, rows gathered by the page table one by one, so pages may end anywhere
// in a tile) and needs no block-wide barrier.  Rows are the M of mma.sync m16n8: the tensor pipe
// has ample room at this ratio, and a warp works alone.
// fp32 caches: products as hi*hi + hi*lo + lo*hi of tf32 halves (about 2^-21 relative), each tile's
// sum added to the running one in fp32; 16-bit caches: q, K, V as stored, and the weights
// 2^(x - m) as a sum of two 16-bit values, so nothing is rounded but the fp32 sums and the output.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "../../include/l2.h"
#include "attn_pages.cuh"
#include "l2_device.cuh"
#include "l2_pages.h"

namespace l2 {

namespace {

constexpr int kStages = 3;     // tiles of a warp's ring
// Fewest tiles a warp takes: below that the parts cost more to write and merge than the
// parallel reading gains.
constexpr int kMinTiles = 4;
constexpr int kTcMinTiles = 4;  // the same for the tensor-core kernel's blocks (tiles of 128 keys)

}  // namespace

namespace {
// Exclusive prefix sum over a block of 1024 threads; buf: 64 ints.
__device__ __forceinline__ int block_scan_1024(int v, int *total, int *buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) buf[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = buf[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        buf[32 + lane] = w;
    }
    __syncthreads();
    const int before = warp ? buf[32 + warp - 1] : 0;
    *total = buf[63];
    __syncthreads();
    return before + x - v;
}
}  // namespace

// One block: lengths of the sources and the numbering of their tiles and items.
// With p.tc the whole tiles of a prefix that serves more than 16 pairs go to the tensor-core kernel.
__global__ void __launch_bounds__(1024) attn_pages_plan_kernel(const PagesAttn p, int tile_keys, int num_sms) {
    __shared__ int part[1][64], minlen[kPagesMaxCall], mintc[kPagesMaxCall], gstart[kPagesMaxCall + 1], len_s[kPagesMaxCall];
    const int i = threadIdx.x;
    const int S = p.G + p.B;
    const Plan pl = plan_of(p.plan, S, p.G);
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    pdl_launch_dependents();
    bool bad = false;
    int len = 0;
    if (i < p.B) {
        const int s = p.seqs ? p.seqs[i] : i;
        bad = s < 0 || s >= p.n_seqs;
        if (!bad) len = p.lens[s];
        bad |= len < 0 || len > (long long)p.max_pages * p.page_size;
    }
    len_s[i] = len;
    if (i <= p.G) {
        const int a = p.G ? p.group_starts[i] : 0;
        bad |= p.G && ((i == 0 && a != 0) || (i == p.G && a != p.B) || a < 0 || a > p.B);
        gstart[i] = a;
    }
    if (i == 0 && p.G == kPagesMaxCall) {  // one entry more than threads
        gstart[p.G] = p.group_starts[p.G];
        bad |= gstart[p.G] != p.B;
    }
    __syncthreads();
    int P = 0, r0 = 0, rows = 0;
    if (i < p.G) {
        r0 = gstart[i];
        rows = gstart[i + 1] - r0;
        P = p.prefix_lens[i];
        bad |= rows < 0 || P < 0;
    }
    if (__syncthreads_or(bad)) {
        if (i == 0) {
            atomicOr(p.err, L2_PAGES_ERR_ARGS);
            pl.hdr[kHdrCost] = pl.hdr[kHdrTcTiles] = 0;
            pl.hdr[kHdrWarps] = pl.hdr[kHdrTcCtas] = 1;
            pl.hdr[kHdrOk] = 0;
        }
        return;
    }
    // a row alone has nothing to share: all its keys are its own
    if (i < p.G) minlen[i] = rows < 2 ? 0 : P;
    __syncthreads();
    if (p.G && i < p.B) {
        int lo = 0, hi = p.G;  // the group of the row: the last that starts at or before it
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            gstart[m] <= i ? lo = m : hi = m;
        }
        atomicMin(&minlen[lo], len);
    }
    __syncthreads();
    // prefixes worth it go to the tensor cores in whole tiles of 128 keys; what is left of them stays here
    int tc_tiles = 0, tc_rows = 0;
    if (p.G) {
        const int n = rows * gq, full = i < p.G && p.tc && n > kM ? minlen[i] / kTcKeys : 0;
        const int tiles = full * tc_runs(n) * p.n_kv_heads, prows = full ? tc_head_rows(n) * p.n_kv_heads : 0;
        const int tb = block_scan_1024(tiles, &tc_tiles, part[0]), rb = block_scan_1024(prows, &tc_rows, part[0]);
        if (i < p.G) {
            pl.tc_t0[i] = tb;
            pl.tc_kt[i] = full;
            pl.tc_r0[i] = rb;
            mintc[i] = full * kTcKeys;
        }
        __syncthreads();
    }
    // sources in blocks of 1024: G prefixes, then B sequences
    int tiles_before = 0, items_before = 0;
    for (int s0 = 0; s0 < S; s0 += 1024) {
        const int s = s0 + i;
        int key0 = 0, key1 = 0, row0 = 0, n = 0;
        if (s < p.G) {
            key0 = mintc[s];
            key1 = minlen[s];
            row0 = gstart[s];
            n = gstart[s + 1] - row0;
        } else if (s < S) {
            row0 = s - p.G;
            n = 1;
            key1 = len_s[row0];
            int lo = 0, hi = p.G;
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                gstart[m] <= row0 ? lo = m : hi = m;
            }
            key0 = p.G ? minlen[lo] : 0;
        }
        const int kt = s < S ? cdiv(key1 - key0, tile_keys) : 0;
        const int items = kt > 0 ? cdiv(n * gq, kM) * p.n_kv_heads : 0;
        const int cost = tile_cost(p.dtype, min(n * gq, kM));
        int tiles_here, items_here;
        const int a = block_scan_1024(items * kt * cost, &tiles_here, part[0]), b = block_scan_1024(items, &items_here, part[0]);
        if (s < S) {
            pl.t0[s] = tiles_before + a;
            pl.cost[s] = cost;
            pl.i0[s] = items_before + b;
            pl.kt[s] = kt;
            pl.key0[s] = key0;
            pl.key1[s] = key1;
            pl.row0[s] = row0;
            pl.rows[s] = n;
        }
        tiles_before += tiles_here;
        items_before += items_here;
    }
    if (i == 0) {
        pl.t0[S] = tiles_before;
        pl.i0[S] = items_before;
        pl.hdr[kHdrCost] = tiles_before;
        pl.hdr[kHdrTcTiles] = tc_tiles;
        pl.hdr[kHdrTcCtas] = max(1, min(num_sms, cdiv(tc_tiles, kTcMinTiles)));
        if (p.G) pl.tc_t0[p.G] = tc_tiles;
        pl.hdr[kHdrWarps] = max(1, min(num_sms * kWalkWarps, cdiv(tiles_before, kMinTiles * kCostUnit)));
        pl.hdr[kHdrOk] = 1;
    }
}

namespace {

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}

struct TBf16 {
    static __device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t v) { return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v)); }
};
struct TF16 {
    static __device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        const __half2 v = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
};

// Tile shape: HS the head size padded to 64 or 128; K and V of a tile's keys take 8 KB.
template <int HS>
struct Shape {
    static constexpr int KT = HS == 128 ? 16 : 32;
    static constexpr int C = HS * 2 / 16;         // 16-byte words a row
    static constexpr int kRow = HS * 2;
    static constexpr int kStage = 2 * KT * kRow;  // K then V
    static constexpr int kSmem = kWalkWarps * kStages * kStage;
};
// Word c of row r sits at word c ^ swz(r): the eight rows that one ldmatrix phase reads fall into
// different banks.
__device__ __forceinline__ int swz(int r) { return r & 7; }

}  // namespace

// The warps' walk (see the head of the file).
template <typename T, int HS>
__global__ void __launch_bounds__(kWalkWarps * 32, 1) attn_pages_kernel(const PagesAttn p) {
    using Sh = Shape<HS>;
    constexpr int KT = Sh::KT, C = Sh::C, NT = KT / 8;  // NT: n8 tiles of keys
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
    const int wid = walker_id();
    const uint32_t ring = smem_u32(smem) + (threadIdx.x >> 5) * (kStages * Sh::kStage);
    const int S = p.G + p.B;
    const Plan pl = plan_of(p.plan, S, p.G);
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    pdl_launch_dependents();
    pdl_wait();
    const int T_all = pl.hdr[kHdrCost], W = pl.hdr[kHdrWarps];
    if (wid >= W) return;
    const int x0 = first_of(wid, T_all, W), x1 = first_of(wid + 1, T_all, W);
    if (x0 >= x1) return;
    int src = warp_find(pl.t0, S + 1, x0), x = x0;
    const int words = p.head_size / 8;  // 16-byte words of a row that exist

    WalkItem w;
    while (walk_item(p, pl, src, x, x1, gq, w)) {
        const char *kb = p.k + w.kvh * p.head_stride, *vb = p.v + w.kvh * p.head_stride;
        // this lane's key of tile i of the item's share
        auto key_of = [&](int i) { return lane < KT && i < w.n_tiles ? w.key0 + (w.k_first + i) * KT + lane : w.key1; };
        auto fetch = [&](int i, int page) {
            const int stage = i % kStages;
            const long long off = walk_place(p, w, key_of(i), page);
            const uint32_t ks = ring + stage * Sh::kStage, vs = ks + KT * Sh::kRow;
            constexpr int RP = C >= 32 ? 1 : 32 / C;  // rows one instruction covers
            const int c = lane % C, rr = C >= 32 ? 0 : lane / C;
#pragma unroll
            for (int r0 = 0; r0 < KT; r0 += RP) {
                const int r = r0 + rr;
                const long long o = __shfl_sync(0xffffffffu, off, r);
                const bool on = o >= 0 && c < words;
                const uint32_t d = r * Sh::kRow + ((c ^ swz(r)) << 4);
                const long long so = on ? o + (c << 4) : 0;
                cp_async16(ks + d, kb + so, on);
                cp_async16(vs + d, vb + so, on);
            }
            cp_commit();
        };

        const int n_tiles = w.n_tiles, k_first = w.k_first;
        int page = walk_page(p, w, key_of(0)), next = walk_page(p, w, key_of(1));
        // fill the ring
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            fetch(s, page);
            page = next;
            next = walk_page(p, w, key_of(s + 2));
        }

        const char *qa = walk_query(p, w, g4, gq), *qb = walk_query(p, w, g4 + 8, gq);
        float m_run[2] = {-CUDART_INF_F, -CUDART_INF_F}, l_run[2] = {0.f, 0.f};
        float o[HS / 8][4];
#pragma unroll
        for (int i = 0; i < HS / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        // 16-bit: the A fragments of all K steps; fp32: the lane's query values
        constexpr int QR = HS / 16 * 4;
        uint32_t qf[QR];
#pragma unroll
        for (int ks = 0; ks < HS / 16; ++ks) {
            const int d0 = ks * 16 + 2 * t4, d1 = d0 + 8;
            qf[4 * ks] = qa && d0 < p.head_size ? *reinterpret_cast<const uint32_t *>(qa + 2 * d0) : 0u;
            qf[4 * ks + 1] = qb && d0 < p.head_size ? *reinterpret_cast<const uint32_t *>(qb + 2 * d0) : 0u;
            qf[4 * ks + 2] = qa && d1 < p.head_size ? *reinterpret_cast<const uint32_t *>(qa + 2 * d1) : 0u;
            qf[4 * ks + 3] = qb && d1 < p.head_size ? *reinterpret_cast<const uint32_t *>(qb + 2 * d1) : 0u;
        }
    

#pragma unroll 1
        for (int it = 0; it < n_tiles; ++it) {
            cp_wait<kStages - 2>();
            __syncwarp();
            // the next tile goes into the stage read one step ago
            if (it + kStages - 1 < n_tiles) {
                fetch(it + kStages - 1, page);
                page = next;
                next = walk_page(p, w, key_of(it + kStages + 1));
            } else {
                cp_commit();
            }
            const uint32_t ks_base = ring + (it % kStages) * Sh::kStage, vs_base = ks_base + KT * Sh::kRow;
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[n][j] = 0.f;
            // lane's ldmatrix row: key (lane & 7) of the n8 tile, word 2 kpair + lane / 8
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int key = 8 * n + (lane & 7);
#pragma unroll
                for (int c = 0; c < C; c += 4) {
                    uint32_t b[4];
                    ldsm4(ks_base + key * Sh::kRow + (((c + (lane >> 3)) ^ swz(key)) << 4), b);
                    T::mma(s[n], qf + 2 * c, b[0], b[1]);
                    T::mma(s[n], qf + 2 * c + 4, b[2], b[3]);
                }
            }
        
            // scale, mask keys past the end, running max
            const int left = w.key1 - w.key0 - (k_first + it) * KT;
            float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = 8 * n + 2 * t4 + (j & 1);
                    s[n][j] = key < left ? s[n][j] * p.scale_log2 : -CUDART_INF_F;
                    mx[j >> 1] = fmaxf(mx[j >> 1], s[n][j]);
                }
            float corr[2], base[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
                const float mn = fmaxf(m_run[r], mx[r]);
                base[r] = mn == -CUDART_INF_F ? 0.f : mn;  // only -inf so far: weights 0, not NaN
                corr[r] = exp2f(m_run[r] - base[r]);
                m_run[r] = mn;
            }
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[n][j] = exp2f(s[n][j] - base[j >> 1]);
                    sum[j >> 1] += s[n][j];
                }
            l_run[0] = l_run[0] * corr[0] + sum[0];
            l_run[1] = l_run[1] * corr[1] + sum[1];
#pragma unroll
            for (int i = 0; i < HS / 8; ++i) {
                o[i][0] *= corr[0];
                o[i][1] *= corr[0];
                o[i][2] *= corr[1];
                o[i][3] *= corr[1];
            }
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk) {
                // weights as A fragments: hi and what it leaves
                uint32_t ph[4], plo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = s[2 * kk + (j >> 1)][2 * (j & 1)], y = s[2 * kk + (j >> 1)][2 * (j & 1) + 1];
                    ph[j] = T::pack(x, y);
                    const float2 back = T::unpack(ph[j]);
                    plo[j] = T::pack(x - back.x, y - back.y);
                }
                const int key = 16 * kk + (lane & 15);
#pragma unroll
                for (int c = 0; c < C; c += 2) {
                    uint32_t b[4];
                    ldsm4t(vs_base + key * Sh::kRow + (((c + (lane >> 4)) ^ swz(key)) << 4), b);
                    T::mma(o[c], ph, b[0], b[1]);
                    T::mma(o[c], plo, b[0], b[1]);
                    T::mma(o[c + 1], ph, b[2], b[3]);
                    T::mma(o[c + 1], plo, b[2], b[3]);
                }
            }
        
            __syncwarp();  // the stage is read before the next fetch into it
        }
        cp_wait<0>();
        __syncwarp();
        // the part: (m, l) and the sums of the item's pairs
        const int slot = pl.i0[w.src] + w.item + wid;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float l = l_run[r];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int mi = g4 + 8 * r;
            if (!(r ? qb : qa) || slot >= p.max_parts) continue;
            if (t4 == 0) reinterpret_cast<float2 *>(p.ws_ml)[(size_t)slot * kM + mi] = make_float2(m_run[r], l);
            float *dst = p.ws_acc + ((size_t)slot * kM + mi) * p.head_size;
#pragma unroll
            for (int i = 0; i < HS / 8; ++i) {
                const int d = 8 * i + 2 * t4;
                if (d < p.head_size) *reinterpret_cast<float2 *>(dst + d) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
            }
        
        }
    }
}

namespace {
constexpr int kMergeThreads = 128;

template <typename T>
__device__ __forceinline__ void store_out(char *o, int d, float4 v);
template <>
__device__ __forceinline__ void store_out<float>(char *o, int d, float4 v) {
    *reinterpret_cast<float4 *>(o + 4 * d) = v;
}
template <>
__device__ __forceinline__ void store_out<TBf16>(char *o, int d, float4 v) {
    *reinterpret_cast<uint2 *>(o + 2 * d) = make_uint2(TBf16::pack(v.x, v.y), TBf16::pack(v.z, v.w));
}
template <>
__device__ __forceinline__ void store_out<TF16>(char *o, int d, float4 v) {
    *reinterpret_cast<uint2 *>(o + 2 * d) = make_uint2(TF16::pack(v.x, v.y), TF16::pack(v.z, v.w));
}
}  // namespace

// One block per (row, query head): its prefix's parts, then its own, merged in key order by four warps
// (part i goes to warp i % 4) and then over the warps in order.
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) attn_pages_merge_kernel(const PagesAttn p) {
    __shared__ float sm[4], sl[4];
    __shared__ float4 sa[4][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / p.n_heads, h = blockIdx.x - b * p.n_heads;
    const int S = p.G + p.B;
    const Plan pl = plan_of(p.plan, S, p.G);
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    const int kvh = (int)((long long)h * p.n_kv_heads / p.n_heads), j = h - first_head(kvh, p.n_heads, p.n_kv_heads);
    const int d = 4 * lane;
    const bool on = d < p.head_size;
    pdl_wait();
    if (!pl.hdr[kHdrOk]) return;
    const int T_all = pl.hdr[kHdrCost], W = pl.hdr[kHdrWarps];
    int grp = -1;
    if (p.G) {
        int lo = 0, hi = p.G;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            p.group_starts[m] <= b ? lo = m : hi = m;
        }
        grp = lo;
    }
    float m = -CUDART_INF_F, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    bool any = false;
    int seen = 0;
    // one part into the warp's running (m, l, a); a part without keys has m = -inf
    auto take = [&](float2 ml, const float *acc) {
        if (ml.x == -CUDART_INF_F && ml.y == 0.f) return;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) v = *reinterpret_cast<const float4 *>(acc + d);
        const float mn = fmaxf(m, ml.x), base = mn == -CUDART_INF_F ? 0.f : mn;
        const float c0 = exp2f(m - base), c1 = exp2f(ml.x - base);
        a.x = a.x * c0 + v.x * c1;
        a.y = a.y * c0 + v.y * c1;
        a.z = a.z * c0 + v.z * c1;
        a.w = a.w * c0 + v.w * c1;
        l = l * c0 + ml.y * c1;
        m = mn;
    };
    if (grp >= 0 && pl.tc_kt[grp]) {
        const int kt = pl.tc_kt[grp], n = pl.rows[grp] * gq, mi = (b - pl.row0[grp]) * gq + j;
        const int run = mi / (2 * kTcRows), r = mi - run * 2 * kTcRows, rows = min(2 * kTcRows, n - run * 2 * kTcRows);
        const int u0 = pl.tc_t0[grp] + (kvh * tc_runs(n) + run) * kt;
        const int Tt = pl.hdr[kHdrTcTiles], Wt = pl.hdr[kHdrTcCtas];
        const int w0 = walker_of(u0, Tt, Wt), w1 = walker_of(u0 + kt - 1, Tt, Wt);
        const int base = pl.tc_r0[grp] + kvh * tc_head_rows(n) + run * 2 * kTcRows + r;
        const int per = rows > kTcRows ? 1 : 2;  // parts a walker leaves of this row
        any = true;
        for (int e = warp; e < (w1 - w0 + 1) * per; e += 4) {
            const int w = w0 + e / per, sl2 = e - (w - w0) * per;
            const size_t at = (size_t)(base + 2 * kTcRows * w + sl2 * rows);
            take(reinterpret_cast<const float2 *>(p.tc_ml)[at], p.tc_acc + at * p.head_size);
        }
        seen = ((w1 - w0 + 1) * per) & 3;
    }
    for (int which = 0; which < 2; ++which) {
        const int s = which ? p.G + b : grp;
        if (s < 0) continue;
        const int kt = pl.kt[s];
        if (kt == 0) continue;
        any = true;
        const int mi = (b - pl.row0[s]) * gq + j, tiles_m = cdiv(pl.rows[s] * gq, kM);
        const int item = kvh * tiles_m + mi / kM;
        const int cost = pl.cost[s], u0 = pl.t0[s] + item * kt * cost;
        const int w0 = walker_of(u0, T_all, W), w1 = walker_of(u0 + (kt - 1) * cost, T_all, W);
        const int slot0 = pl.i0[s] + item;
        for (int w = w0 + ((warp - seen) & 3); w <= w1; w += 4) {
            // a walker whose range is narrower than a tile may hold none of it
            const int lo = max(u0, first_of(w, T_all, W)), hi = min(u0 + kt * cost, first_of(w + 1, T_all, W));
            if (cdiv(lo - u0, cost) >= cdiv(hi - u0, cost)) continue;
            const size_t at = (size_t)(slot0 + w) * kM + (mi % kM);
            take(reinterpret_cast<const float2 *>(p.ws_ml)[at], p.ws_acc + at * p.head_size);
        }
        seen = (seen + (w1 - w0 + 1)) & 3;
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    sa[warp][lane] = a;
    __syncthreads();
    if (warp) return;
    for (int w = 1; w < 4; ++w) {
        const float mn = fmaxf(m, sm[w]), base = mn == -CUDART_INF_F ? 0.f : mn;
        const float c0 = exp2f(m - base), c1 = exp2f(sm[w] - base);
        const float4 v = sa[w][lane];
        a.x = a.x * c0 + v.x * c1;
        a.y = a.y * c0 + v.y * c1;
        a.z = a.z * c0 + v.z * c1;
        a.w = a.w * c0 + v.w * c1;
        l = l * c0 + sl[w] * c1;
        m = mn;
    }
    // no keys at all: zeros, and a sum of nothing; all scores -inf: 0 / 0, as the formula has it
    const float inv = any ? 1.0f / l : 0.f;
    if (on)
        store_out<T>(p.out + (long long)b * p.o_row + (long long)h * p.o_head, d,
                     any ? make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f));
    if (p.lse && lane == 0) p.lse[(size_t)b * p.n_heads + h] = any ? (m + log2f(l)) * 0.6931471805599453f : -CUDART_INF_F;
}

namespace {

template <typename T, int HS>
cudaError_t launch_walk(const PagesAttn &p, int grid, cudaLaunchConfig_t cfg) {
    using Sh = Shape<HS>;
    auto fn = attn_pages_kernel<T, HS>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kWalkWarps * 32);
    cfg.dynamicSmemBytes = Sh::kSmem;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

int tile_keys(int dtype, int hs) {
    return dtype == L2_F32 ? attn_pages_f32_tile(hs) : hs <= 64 ? Shape<64>::KT : Shape<128>::KT;
}

int max_items(int B, int G, int n_heads, int n_kv_heads) {
    // prefix tiles: sum over groups of ceil(rows gq / 16) <= (B gq) / 16 + G
    const long long gq = heads_per_kv(n_heads, n_kv_heads);
    const long long pre = G ? (B * gq) / kM + G : 0, own = B * ((gq + kM - 1) / kM);
    return (int)((pre + own) * n_kv_heads);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Rows of the tensor-core kernel's parts: each run at most twice its pairs, and 256 a block.
size_t tc_part_rows(int B, int n_heads, int n_kv_heads, int num_sms) {
    return 2 * (size_t)B * heads_per_kv(n_heads, n_kv_heads) * n_kv_heads + 2 * kTcRows * (size_t)(num_sms + 1);
}

// The workspace's parts, in order.
struct WsLayout {
    size_t plan, ml, acc, tc_ml, tc_acc, bytes, parts;
};
WsLayout ws_layout(int B, int G, int n_heads, int n_kv_heads, int head_size, int num_sms) {
    WsLayout w;
    w.parts = (size_t)max_items(B, G, n_heads, n_kv_heads) + (size_t)num_sms * kWalkWarps;
    const size_t tc = G ? tc_part_rows(B, n_heads, n_kv_heads, num_sms) : 0;
    w.plan = 0;
    w.ml = w.plan + align256(plan_ints(B + G, G) * 4);
    w.acc = w.ml + align256(w.parts * kM * 8);
    w.tc_ml = w.acc + align256(w.parts * kM * head_size * 4);
    w.tc_acc = w.tc_ml + align256(tc * 8);
    w.bytes = w.tc_acc + align256(tc * head_size * 4);
    return w;
}

}  // namespace

size_t pages_attn_ws_bytes(int B, int G, int n_heads, int n_kv_heads, int head_size, int num_sms) {
    return ws_layout(B, G, n_heads, n_kv_heads, head_size, num_sms).bytes;
}

cudaError_t launch_pages_attn(PagesAttn p, void *ws, int num_sms, cudaStream_t s) {
    const WsLayout w = ws_layout(p.B, p.G, p.n_heads, p.n_kv_heads, p.head_size, num_sms);
    char *base = static_cast<char *>(ws);
    p.plan = reinterpret_cast<int *>(base + w.plan);
    p.ws_ml = reinterpret_cast<float *>(base + w.ml);
    p.ws_acc = reinterpret_cast<float *>(base + w.acc);
    p.tc_ml = reinterpret_cast<float *>(base + w.tc_ml);
    p.tc_acc = reinterpret_cast<float *>(base + w.tc_acc);
    p.max_parts = (int)w.parts;
    // a prefix that serves at most 16 pairs or is shorter than a tile gains nothing there
    p.tc = p.G && p.B * heads_per_kv(p.n_heads, p.n_kv_heads) > kM && attn_pages_tc_supported(p);
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cudaError_t e = cudaLaunchKernelEx(&cfg, attn_pages_plan_kernel, p, tile_keys(p.dtype, p.head_size), num_sms);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
    if (p.tc && (e = launch_attn_pages_tc(p, num_sms, cfg)) != cudaSuccess) return e;
    const int hs = p.head_size;
    if (p.dtype == L2_F32)
        e = launch_attn_pages_f32(p, num_sms, cfg);
    else if (p.dtype == L2_BF16)
        e = hs <= 64 ? launch_walk<TBf16, 64>(p, num_sms, cfg) : launch_walk<TBf16, 128>(p, num_sms, cfg);
    else
        e = hs <= 64 ? launch_walk<TF16, 64>(p, num_sms, cfg) : launch_walk<TF16, 128>(p, num_sms, cfg);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(p.B * p.n_heads);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    if (p.dtype == L2_F32) return cudaLaunchKernelEx(&cfg, attn_pages_merge_kernel<float>, p);
    if (p.dtype == L2_BF16) return cudaLaunchKernelEx(&cfg, attn_pages_merge_kernel<TBf16>, p);
    return cudaLaunchKernelEx(&cfg, attn_pages_merge_kernel<TF16>, p);
}

}  // namespace l2
