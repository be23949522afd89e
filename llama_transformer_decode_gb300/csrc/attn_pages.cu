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
#include "attn_plan.cuh"
#include "l2_device.cuh"
#include "l2_pages.h"

namespace l2 {

namespace {

constexpr int kStages = 3;     // tiles of a warp's ring

}  // namespace

// The plan as a kernel of its own, for calls of more sources than a block plans for itself.
__global__ void __launch_bounds__(kPagesMaxCall) attn_pages_plan_kernel(const PagesAttn p) {
    __shared__ PlanScratch<kPagesMaxCall, kPagesMaxCall> sc;
    pdl_launch_dependents();
    plan_build<kPagesMaxCall, kPagesMaxCall>(p, plan_of(p.plan, p.B, p.G), sc, true);
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
    static constexpr int kRings = kWalkWarps * kStages * kStage;
    static constexpr int kSmem = kRings + (int)kPlanSmem;
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
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    pdl_launch_dependents();
    if (p.wait_first) pdl_wait();
    const Plan pl = plan_here<kWalkWarps * 32>(p, smem + Sh::kRings, smem, blockIdx.x == 0);
    const int T_all = pl.hdr[kHdrCost], W = pl.hdr[kHdrWarps];
    const int x0 = wid < W ? first_of(wid, T_all, W) : 0, x1 = wid < W ? first_of(wid + 1, T_all, W) : 0;
    const int words = p.head_size / 8;  // 16-byte words of a row that exist
    int src = 0, x = x0, done = 0;
    WalkAhead<KT> ahead;
    if (x0 < x1) {
        src = warp_find(&pl.src[0].t0, sizeof(Source) / 4, p.G + p.B + 1, x0);
        ahead.start(p, pl, src, x0, x1, gq);
        for (int s = 0; s < kStages - 1; ++s) {
            const uint32_t ks = ring + s * Sh::kStage;
            walk_copy<KT, Sh::kRow>(p, pl, ahead, x1, gq, words, ks, ks + KT * Sh::kRow, swz);
        }
    }

    WalkItem w;
    while (walk_item(p, pl, src, x, x1, gq, w)) {
        const int n_tiles = w.n_tiles, k_first = w.k_first;
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
        for (int it = 0; it < n_tiles; ++it, ++done) {
            cp_wait<kStages - 2>();
            __syncwarp();
            // the next tile goes into the stage read one step ago
            const uint32_t nx = ring + ((done + kStages - 1) % kStages) * Sh::kStage;
            walk_copy<KT, Sh::kRow>(p, pl, ahead, x1, gq, words, nx, nx + KT * Sh::kRow, swz);
            const uint32_t ks_base = ring + (done % kStages) * Sh::kStage, vs_base = ks_base + KT * Sh::kRow;
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
        // the part: (m, l) and the sums of the item's pairs
        const int slot = w.slot + wid;
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
    cp_wait<0>();
    // the merge waits for this kernel alone: it ends after the tensor-core kernel before it
    if (p.tc && threadIdx.x == 0) pdl_wait();
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

// Parts of one (row, head) that a source's walkers left.
struct PartRange {
    int u0, kt, cost, w0, n, slot, pair;
};
}  // namespace

// One warp per (row, query head): the parts of its prefix and of its own keys, in key order.  Lanes take a part each
// for (m, l), so all weights are known after one round of loads; then the warp adds the parts' sums, LP
// lanes to a part.
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) attn_pages_merge_kernel(const PagesAttn p) {
    const int lane = threadIdx.x & 31;
    const int bh = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
    const int b = bh / p.n_heads, h = bh - b * p.n_heads;
    const Plan pl = plan_of(p.plan, p.B, p.G);
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    const int kvh = (int)((long long)h * p.n_kv_heads / p.n_heads), j = h - first_head(kvh, p.n_heads, p.n_kv_heads);
    pdl_wait();
    if (b >= p.B || !pl.hdr[kHdrOk]) return;
    const int T_all = pl.hdr[kHdrCost], W = pl.hdr[kHdrWarps];
    const int grp = p.G ? pl.group[b] : 0;
    auto range = [&](int s) {
        PartRange r = {};
        const int4 a = *reinterpret_cast<const int4 *>(&pl.src[s].t0), c = *reinterpret_cast<const int4 *>(&pl.src[s].key0);
        if (a.z) {
            const int mi = (b - c.z) * gq + j, item = kvh * cdiv(c.w * gq, kM) + mi / kM;
            r.kt = a.z;
            r.cost = a.w;
            r.u0 = a.x + item * a.z * a.w;
            r.w0 = walker_of(r.u0, T_all, W);
            r.n = walker_of(r.u0 + (a.z - 1) * a.w, T_all, W) - r.w0 + 1;
            r.slot = a.y + item;
            r.pair = mi % kM;
        }
        return r;
    };
    const PartRange own = range(p.G + b);
    PartRange rest = {};
    int tc_n = 0, tc_w0 = 0, tc_base = 0, tc_rows = 0, tc_per = 1;
    if (p.G) {
        rest = range(grp);
        const int kt = pl.tc_kt[grp];
        if (kt) {
            const int row0 = pl.src[grp].row0, n = pl.src[grp].rows * gq, mi = (b - row0) * gq + j;
            const int run = mi / (2 * kTcRows), r = mi - run * 2 * kTcRows;
            const int u0 = pl.tc_t0[grp] + (kvh * tc_runs(n) + run) * kt, Tt = pl.hdr[kHdrTcTiles], Wt = pl.hdr[kHdrTcCtas];
            tc_rows = min(2 * kTcRows, n - run * 2 * kTcRows);
            tc_per = tc_rows > kTcRows ? 1 : 2;  // parts a block leaves of this row
            tc_w0 = walker_of(u0, Tt, Wt);
            tc_n = (walker_of(u0 + kt - 1, Tt, Wt) - tc_w0 + 1) * tc_per;
            tc_base = pl.tc_r0[grp] + kvh * tc_head_rows(n) + run * 2 * kTcRows + r;
        }
    }
    const int n = tc_n + rest.n + own.n;
    const int LP = p.head_size > 64 ? 32 : p.head_size > 32 ? 16 : 8;  // lanes of a part's sums
    const int sub = lane / LP, d = 4 * (lane % LP), per = 32 / LP;
    const bool on = d < p.head_size;
    float m = -CUDART_INF_F, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int e0 = 0; e0 < n; e0 += 32) {
        const int e = e0 + lane;
        float2 ml = make_float2(-CUDART_INF_F, 0.f);
        const float *acc = nullptr;
        if (e < tc_n) {
            const int wi = e / tc_per;
            const size_t at = (size_t)(tc_base + 2 * kTcRows * (tc_w0 + wi) + (e - wi * tc_per) * tc_rows);
            ml = reinterpret_cast<const float2 *>(p.tc_ml)[at];
            acc = p.tc_acc + at * p.head_size;
        } else if (e < n) {
            const bool first = e < tc_n + rest.n;
            const PartRange &r = first ? rest : own;
            const int w = r.w0 + e - tc_n - (first ? 0 : rest.n);
            // a walker whose range is narrower than a tile may hold none of it
            const int lo = max(r.u0, first_of(w, T_all, W)), hi = min(r.u0 + r.kt * r.cost, first_of(w + 1, T_all, W));
            if (cdiv(lo - r.u0, r.cost) < cdiv(hi - r.u0, r.cost)) {
                const size_t at = (size_t)(r.slot + w) * kM + r.pair;
                ml = reinterpret_cast<const float2 *>(p.ws_ml)[at];
                acc = p.ws_acc + at * p.head_size;
            }
        }
        if (ml.x == -CUDART_INF_F && ml.y == 0.f) acc = nullptr;  // a part without keys
        float mn = fmaxf(m, ml.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        const float base = mn == -CUDART_INF_F ? 0.f : mn;
        const float c0 = exp2f(m - base), wt = exp2f(ml.x - base);
        float ls = acc ? ml.y * wt : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        l = l * c0 + ls;
        m = mn;
        a.x *= c0;
        a.y *= c0;
        a.z *= c0;
        a.w *= c0;
        const int cnt = min(32, n - e0);
#pragma unroll 8
        for (int q = 0; q < cnt; q += per) {
            const int from = min(q + sub, 31);
            const float c1 = __shfl_sync(0xffffffffu, wt, from);
            const float *src = reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(acc), from));
            if (q + sub < cnt && src && on) {
                const float4 v = *reinterpret_cast<const float4 *>(src + d);
                a.x = fmaf(v.x, c1, a.x);
                a.y = fmaf(v.y, c1, a.y);
                a.z = fmaf(v.z, c1, a.z);
                a.w = fmaf(v.w, c1, a.w);
            }
        }
    }
    for (int o = 16; o >= LP; o >>= 1) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
        a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    }
    // no keys at all: zeros, and a sum of nothing; all scores -inf: 0 / 0, as the formula has it
    const float inv = n ? 1.0f / l : 0.f;
    if (on && sub == 0)
        store_out<T>(p.out + (long long)b * p.o_row + (long long)h * p.o_head, d,
                     n ? make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f));
    if (p.lse && lane == 0) p.lse[(size_t)b * p.n_heads + h] = n ? (m + log2f(l)) * 0.6931471805599453f : -CUDART_INF_F;
}

namespace {

template <typename T, int HS>
cudaError_t launch_walk(const PagesAttn &p, cudaLaunchConfig_t cfg) {
    auto fn = attn_pages_kernel<T, HS>;
    static DeviceOnce once;
    cudaError_t e = once.smem(reinterpret_cast<const void *>(fn), Shape<HS>::kSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(p.num_sms);
    cfg.blockDim = dim3(kWalkWarps * 32);
    cfg.dynamicSmemBytes = Shape<HS>::kSmem;
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
    w.ml = w.plan + align256(plan_bytes(B, G));
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

// Kernels of a call, each after the first launched as its predecessor's dependent: [plan] [tensor cores] warps, merge.
cudaError_t launch_pages_attn(PagesAttn p, void *ws, int num_sms, cudaStream_t s) {
    const WsLayout w = ws_layout(p.B, p.G, p.n_heads, p.n_kv_heads, p.head_size, num_sms);
    char *base = static_cast<char *>(ws);
    p.plan = reinterpret_cast<int *>(base + w.plan);
    p.ws_ml = reinterpret_cast<float *>(base + w.ml);
    p.ws_acc = reinterpret_cast<float *>(base + w.acc);
    p.tc_ml = reinterpret_cast<float *>(base + w.tc_ml);
    p.tc_acc = reinterpret_cast<float *>(base + w.tc_acc);
    p.max_parts = (int)w.parts;
    p.num_sms = num_sms;
    p.tile_keys = tile_keys(p.dtype, p.head_size);
    // a prefix that serves at most 16 pairs or is shorter than a tile gains nothing there
    p.tc = p.G && p.B * heads_per_kv(p.n_heads, p.n_kv_heads) > kM && attn_pages_tc_supported(p);
    p.plan_in_block = p.B + p.G <= kPlanInBlock;
    p.wait_first = !p.plan_in_block && !p.tc;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cudaError_t e = cudaSuccess;
    if (!p.plan_in_block) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(kPagesMaxCall);
        if ((e = cudaLaunchKernelEx(&cfg, attn_pages_plan_kernel, p)) != cudaSuccess) return e;
        cfg.numAttrs = 1;
    }
    if (p.tc) {
        if ((e = launch_attn_pages_tc(p, cfg)) != cudaSuccess) return e;
        cfg.numAttrs = 1;
    }
    const int hs = p.head_size;
    if (p.dtype == L2_F32)
        e = launch_attn_pages_f32(p, cfg);
    else if (p.dtype == L2_BF16)
        e = hs <= 64 ? launch_walk<TBf16, 64>(p, cfg) : launch_walk<TBf16, 128>(p, cfg);
    else
        e = hs <= 64 ? launch_walk<TF16, 64>(p, cfg) : launch_walk<TF16, 128>(p, cfg);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((p.B * p.n_heads + kMergeThreads / 32 - 1) / (kMergeThreads / 32));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    if (p.dtype == L2_F32) return cudaLaunchKernelEx(&cfg, attn_pages_merge_kernel<float>, p);
    if (p.dtype == L2_BF16) return cudaLaunchKernelEx(&cfg, attn_pages_merge_kernel<TBf16>, p);
    return cudaLaunchKernelEx(&cfg, attn_pages_merge_kernel<TF16>, p);
}

}  // namespace l2
