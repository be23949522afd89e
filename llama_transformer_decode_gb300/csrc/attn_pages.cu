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
// Caches of either kind are walked (attn_pages_f32.cu, attn_pages_16.cu); prefixes that serve many pairs go to the tensor
// cores instead, as blocks of the same kernel (attn_pages_tc32.cuh, attn_pages_tc.cuh).  A walking warp keeps its own ring of tiles (cp.async,
// 16-byte words, rows gathered by the page table one by one, so pages may end anywhere in a tile) and needs no
// block-wide barrier; with all warps reading, HBM is the bound.
//
// Here: the plan as a kernel (large calls), the merge, and the launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <type_traits>

#include "../../include/l2.h"
#include "attn_pages.cuh"
#include "attn_plan.cuh"
#include "l2_device.cuh"
#include "l2_pages.h"

namespace l2 {

// The plan as a kernel of its own, for calls of more sources than a block plans for itself and for wide ones.
__global__ void __launch_bounds__(kPagesMaxCall) attn_pages_plan_kernel(const PagesAttn p) {
    __shared__ PlanScratch<kPagesMaxCall, kPagesMaxCall> sc;
    pdl_launch_dependents();
    pdl_wait();
    const Plan pl = plan_of(p.plan, p.B, p.G);
    plan_build<kPagesMaxCall, kPagesMaxCall, true>(p, pl, sc, true);
    plan_rows<kPagesMaxCall>(p, pl, pl.row);
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
__device__ __forceinline__ void store_out<__nv_bfloat16>(char *o, int d, float4 v) {
    reinterpret_cast<__nv_bfloat162 *>(o + 2 * d)[0] = __floats2bfloat162_rn(v.x, v.y);
    reinterpret_cast<__nv_bfloat162 *>(o + 2 * d)[1] = __floats2bfloat162_rn(v.z, v.w);
}
template <>
__device__ __forceinline__ void store_out<__half>(char *o, int d, float4 v) {
    reinterpret_cast<__half2 *>(o + 2 * d)[0] = __floats2half2_rn(v.x, v.y);
    reinterpret_cast<__half2 *>(o + 2 * d)[1] = __floats2half2_rn(v.z, v.w);
}

constexpr int kEarly = 8;  // rounds of parts' sums loaded before their weights are known
}  // namespace

// NW warps per (row, query head) take the parts of its prefix and of its own keys in turn.  Lanes take a part each
// for (m, l), so a warp's weights are known after one round of loads; LP lanes take a part's sums, the first kEarly
// rounds of which are loaded beside (m, l).  Then the warps' results are joined in order.
template <typename T, int NW>
__global__ void __launch_bounds__(kMergeThreads) attn_pages_merge_kernel(const PagesAttn p) {
    constexpr bool f32 = std::is_same<T, float>::value;
    constexpr int kRows = kMergeThreads / 32 / NW;  // (row, head) pairs a block
    __shared__ float sm[NW], sl[NW];
    __shared__ float4 sa[NW][32];
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % NW;
    const int bh = blockIdx.x * kRows + (threadIdx.x >> 5) / NW;
    const int b = (int)((unsigned)bh / (unsigned)p.n_heads), h = bh - b * p.n_heads;
    const Plan pl = plan_of(p.plan, p.B, p.G);
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    const int kvh = (int)((unsigned)(h * p.n_kv_heads) / (unsigned)p.n_heads), j = h - first_head(kvh, p.n_heads, p.n_kv_heads);
    const int LP = p.head_size > 64 ? 32 : p.head_size > 32 ? 16 : 8;  // lanes of a part's sums
    const int sub = lane / LP, d = 4 * (lane % LP), at_once = 32 / LP;
    const bool on = d < p.head_size;
    pdl_launch_dependents();
    pdl_wait();
    if (b >= p.B) return;
    const int4 h0 = *reinterpret_cast<const int4 *>(pl.hdr);
    const int per_tc = pl.hdr[kHdrTcPer];
    const int4 *rp = reinterpret_cast<const int4 *>(pl.row + b);
    const int4 ow = rp[0], re = rp[1], tc = rp[2];
    const int gr = rp[3].x, per = h0.y;
    if (!h0.z) return;
    // first walker, parts and first row of the parts of the item that holds pair mi of a source of n pairs
    struct Range {
        int w0, n, row;
    };
    auto range = [&](const int4 &s, int mi, int n) {
        Range r = {};
        if (s.z) {
            const int item = kvh * ((n + kM - 1) / kM) + mi / kM, u0 = s.x + item * (kItemCost + s.z * s.w);
            r.w0 = walker_of(u0, per);
            r.n = walker_of(u0 + tile_place(s.z - 1, kItemCost, s.w), per) - r.w0 + 1;
            r.row = (s.y + item + r.w0) * kM + mi % kM;
        }
        return r;
    };
    const Range own = range(ow, j, gq);
    Range rest = {};
    int tc_n = 0, tc_row = 0, tc_rows = 0, tc_two = 0;
    if (p.G) {
        const int n = tc.w * gq, mi = gr * gq + j;
        rest = range(re, mi, n);
        if (tc.y) {
            const int run = mi / tc_run(f32), cost = tc_cost(n, p.head_size, f32);
            const int u0 = tc.x + (kvh * tc_runs(n, f32) + run) * (kTcItemCost + tc.y * cost), w0 = walker_of(u0, per_tc);
            tc_rows = min(tc_run(f32), n - run * tc_run(f32));
            tc_two = !f32 && tc_rows <= kTcRows;  // two parts of this row a block, tc_rows apart
            tc_n = (walker_of(u0 + tile_place(tc.y - 1, kTcItemCost, cost), per_tc) - w0 + 1) << tc_two;
            tc_row = tc.z + kvh * tc_head_rows(n, f32) + mi + tc_run(f32) * w0;
        }
    }
    const int total = tc_n + rest.n + own.n, n = (total + NW - 1 - warp) / NW;  // parts of the row, of this warp
    // (m, l) and sums of the warp's i-th part
    auto part = [&](int i, const float2 *&ml, const float *&acc) {
        int e = i * NW + warp;
        if (e < tc_n) {
            const size_t at = (size_t)(tc_row + tc_run(f32) * (e >> tc_two) + (tc_two ? (e & 1) * tc_rows : 0));
            ml = reinterpret_cast<const float2 *>(p.tc_ml) + at;
            acc = p.tc_acc + at * p.head_size;
        } else {
            e -= tc_n;
            const size_t at = (size_t)(e < rest.n ? rest.row + e * kM : own.row + (e - rest.n) * kM);
            ml = reinterpret_cast<const float2 *>(p.ws_ml) + at;
            acc = p.ws_acc + at * p.head_size;
        }
    };
    auto sums = [&](int e) {
        const float2 *ml;
        const float *acc;
        part(e, ml, acc);
        return *reinterpret_cast<const float4 *>(acc + d);
    };
    float m = -CUDART_INF_F, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int e0 = 0; e0 < n; e0 += 32) {
        const int e = e0 + lane, cnt = min(32, n - e0);
        float2 ml = make_float2(-CUDART_INF_F, 0.f);
        if (e < n) {
            const float2 *pm;
            const float *acc;
            part(e, pm, acc);
            ml = *pm;
        }
        float4 v[kEarly];
#pragma unroll
        for (int q = 0; q < kEarly; ++q)
            if (on && q * at_once + sub < cnt) v[q] = sums(e0 + q * at_once + sub);
        const bool some = !(ml.x == -CUDART_INF_F && ml.y == 0.f);  // a part without keys has sums of no matter
        float mn = fmaxf(m, ml.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        const float base = mn == -CUDART_INF_F ? 0.f : mn;
        const float c0 = exp2f(m - base), wt = exp2f(ml.x - base);
        float ls = some ? ml.y * wt : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        l = l * c0 + ls;
        m = mn;
        a.x *= c0;
        a.y *= c0;
        a.z *= c0;
        a.w *= c0;
        const unsigned have = __ballot_sync(0xffffffffu, some);
        auto add = [&](int q, const float4 &x, float w) {
            if (on && q < cnt && (have >> q & 1)) {
                a.x = fmaf(x.x, w, a.x);
                a.y = fmaf(x.y, w, a.y);
                a.z = fmaf(x.z, w, a.z);
                a.w = fmaf(x.w, w, a.w);
            }
        };
#pragma unroll
        for (int q = 0; q < kEarly; ++q) {
            const int i = q * at_once + sub;
            add(i, v[q], __shfl_sync(0xffffffffu, wt, i & 31));
        }
#pragma unroll 4
        for (int q = kEarly * at_once; q < cnt; q += at_once) {
            const int i = q + sub;
            const float w = __shfl_sync(0xffffffffu, wt, i & 31);
            if (on && i < cnt) add(i, sums(e0 + i), w);
        }
    }
#pragma unroll
    for (int o = 16; o >= 8; o >>= 1)
        if (o >= LP) {
            a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
            a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
            a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
            a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
        }
    if constexpr (NW > 1) {
        if (sub == 0) sa[warp][lane] = a;
        if (lane == 0) {
            sm[warp] = m;
            sl[warp] = l;
        }
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int w = 1; w < NW; ++w) m = fmaxf(m, sm[w]);
        const float base = m == -CUDART_INF_F ? 0.f : m;
        l = 0.f;
        a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w >= total) break;  // a warp without parts
            const float c = exp2f(sm[w] - base);
            const float4 v = sa[w][lane % LP];
            l = fmaf(sl[w], c, l);
            a.x = fmaf(v.x, c, a.x);
            a.y = fmaf(v.y, c, a.y);
            a.z = fmaf(v.z, c, a.z);
            a.w = fmaf(v.w, c, a.w);
        }
    }
    // no keys at all: zeros, and a sum of nothing; all scores -inf: 0 / 0, as the formula has it
    const float inv = total ? 1.0f / l : 0.f;
    if (on && sub == 0)
        store_out<T>(p.out + (long long)b * p.o_row + (long long)h * p.o_head, d,
                     total ? make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f));
    if (p.lse && lane == 0) p.lse[(size_t)b * p.n_heads + h] = total ? (m + log2f(l)) * 0.6931471805599453f : -CUDART_INF_F;
}

namespace {

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
    w.ml = w.plan + align256(plan_bytes(B, G) + (size_t)B * sizeof(RowPlan));
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

// Kernels of a call: [plan] parts, merge.  Each is launched as a dependent of what is before it in the stream (the first too: its blocks
// come up while that ends, and wait for its end before they read anything).
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
    const bool f32 = p.dtype == L2_F32;
    p.tile_shift = f32 ? attn_pages_f32_shift(p.head_size) : attn_pages_16_shift(p.head_size);
    // whether any prefix of such a call could be one for the tensor cores; the plan decides for each
    p.tc = p.G && tc_worth(p, p.B * heads_per_kv(p.n_heads, p.n_kv_heads), p.max_pages * p.page_size) && (f32 || attn_pages_tc_supported(p));
    p.plan_in_block = p.B + p.G <= kPlanInBlock && !p.wide;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaSuccess;
    if (!p.plan_in_block) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(kPagesMaxCall);
        if ((e = cudaLaunchKernelEx(&cfg, attn_pages_plan_kernel, p)) != cudaSuccess) return e;
    }
    if ((e = f32 ? launch_attn_pages_f32(p, cfg) : launch_attn_pages_16(p, cfg)) != cudaSuccess) return e;
    // few (row, head) pairs: four warps to each, since prefixes then come in many parts (a row of 112 parts: 57 -> 31 us a call);
    // many: one warp to each (2048 pairs of 7 parts: 41 us a call against 46)
    const int pairs = p.B * p.n_heads;
    const bool few = pairs <= 1024;
    cfg.gridDim = dim3(few ? pairs : (pairs + 3) / 4);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    if (f32) return cudaLaunchKernelEx(&cfg, few ? attn_pages_merge_kernel<float, 4> : attn_pages_merge_kernel<float, 1>, p);
    if (p.dtype == L2_BF16)
        return cudaLaunchKernelEx(&cfg, few ? attn_pages_merge_kernel<__nv_bfloat16, 4> : attn_pages_merge_kernel<__nv_bfloat16, 1>, p);
    return cudaLaunchKernelEx(&cfg, few ? attn_pages_merge_kernel<__half, 4> : attn_pages_merge_kernel<__half, 1>, p);
}

}  // namespace l2
