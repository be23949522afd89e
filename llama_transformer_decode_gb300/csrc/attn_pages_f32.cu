// The walk of the paged attention over fp32 caches (see attn_pages.cu for the split into items, tiles and parts).
//
// Products are fp32 FMAs on the CUDA cores.  An item has 1 to 16 (row, head) pairs, so a word of K or V read
// serves at most 16 FMAs: at 4 FMAs a byte an SM needs about 60% of its FMA rate to keep up with HBM, and the
// result is as exact as a plain fp32 sum.  (mma.sync with tf32 halves was built first: three products of
// 16 padded rows each took 252 us where this kernel's figure stands in the table of cases, and
// left 5 times the error of an fp32 sum.)
//
// A warp's tile is KT keys (8 KB of K and V).  Scores: a lane takes A keys by Q pairs over every D-th
// 16-byte word of the head, so each word of K read from shared memory meets Q queries and each query word A
// keys; the D lanes of a block of scores add up by a butterfly that leaves each lane its share of them.
// The scores go through shared memory once: 32 / R lanes to a pair take the softmax (running max and
// sum), then every lane holds one 16-byte word of the head for all R pairs and adds weight times V.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "../../include/l2.h"
#include "attn_pages.cuh"
#include "attn_plan.cuh"
#include "l2_device.cuh"
#include "l2_pages.h"

namespace l2 {

namespace {

constexpr int kStagesF = 2;  // tiles of a warp's ring; shared memory holds the queries of 16 pairs beside it

template <int HS>
struct ShapeF {
    static constexpr int KT = HS == 128 ? 8 : HS == 64 ? 16 : 32;
    static constexpr int C = HS / 4;              // 16-byte words a row
    static constexpr int kRow = HS * 4;
    static constexpr int kStage = 2 * KT * kRow;  // K then V
    static constexpr int kQ = kM * kRow;          // queries
    static constexpr int kS = KT * kM * 4;        // scores, then weights [key][pair]
    static constexpr int kWarp = kStagesF * kStage + kQ + kS + kM * 4;
    static constexpr int kSmem = kWalkWarps * kWarp + (int)kPlanSmem;
};

// Word c of row r sits at word c ^ swzf(r): two rows by four words, or one row by eight, fall into different banks.
__device__ __forceinline__ int swzf(int r) { return ((r & 1) << 2) | ((r >> 1) & 3); }

// How a warp's lanes divide the scores of KT keys by R pairs: D lanes along the head, A keys and Q pairs a lane.
template <int KT, int R>
struct Split {
    static constexpr int D = R <= 4 ? 4 : KT == 8 ? 8 : (KT == 32 && R == 16) ? 2 : 4;
    static constexpr int Q = R <= 8 ? R : 8;
    static constexpr int A = KT * (R / Q) * D / 32;
    static_assert(A >= 1 && (KT / A) * (R / Q) * D == 32, "the lanes must cover the scores once");
};

// Adds v[0 .. N) over the D lanes whose numbers differ in their low bits; each lane ends with N / D of the sums (all
// of them when there are fewer than lanes), from index *first on.
template <int N, int D>
__device__ __forceinline__ void lane_sums(float *v, int lane, int &first) {
    first = 0;
    if constexpr (D > 1) {
        constexpr int H = D / 2;
        if constexpr (N > 1) {
            const bool up = lane & H;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float keep = up ? v[i + N / 2] : v[i], send = up ? v[i] : v[i + N / 2];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, H);
            }
            int f;
            lane_sums<N / 2, H>(v, lane, f);
            first = f + (up ? N / 2 : 0);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], H);
            lane_sums<1, H>(v, lane, first);
        }
    }
}
template <int N, int D>
constexpr int kKept = N >= D ? N / D : 1;

// One item of at most R pairs, its first two tiles already under way; done: tiles the warp has computed before.
template <int HS, int R>
__device__ __forceinline__ void walk_f32(const PagesAttn &p, const Plan &pl, const WalkItem &w, WalkAhead<ShapeF<HS>::KT> &ahead, int x1,
                                         int wid, int gq, unsigned char *ring, int done) {
    using Sh = ShapeF<HS>;
    constexpr int KT = Sh::KT, C = Sh::C;
    using Sp = Split<KT, R>;
    constexpr int A = Sp::A, Q = Sp::Q, D = Sp::D;
    const int lane = threadIdx.x & 31;
    unsigned char *qs = ring + kStagesF * Sh::kStage;
    float *ss = reinterpret_cast<float *>(qs + Sh::kQ), *cs = ss + Sh::kS / 4;
    auto word = [](const unsigned char *a) { return *reinterpret_cast<const float4 *>(a); };
    const int words = p.head_size / 4;
    // queries
    for (int e = lane; e < R * C; e += 32) {
        const int i = e / C, c = e - i * C;
        const char *q = walk_query(p, w, i, gq);
        const float4 v = q && c < words ? reinterpret_cast<const float4 *>(q)[c] : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(qs + i * Sh::kRow + (c << 4)) = v;
    }

    // scores: D lanes along the head, then keys, then pairs
    const int d = lane % D, kg = (lane / D) % (KT / A), rg = lane / D / (KT / A);
    // softmax: LP lanes to pair sr
    constexpr int LP = 32 / R;
    const int sr = lane / LP, sk = lane % LP;
    float m_run = -CUDART_INF_F, l_run = 0.f;
    // sums: word vc of the head, keys vk, vk + VK, ..
    constexpr int VK = 32 / C;
    const int vc = lane % C, vk = lane / C;
    float2 acc[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = make_float2(0.f, 0.f);

#pragma unroll 1
    for (int it = 0; it < w.n_tiles; ++it) {
        cp_wait<1>();
        __syncwarp();
        unsigned char *ks = ring + ((done + it) & 1) * Sh::kStage, *vs = ks + KT * Sh::kRow;
        {
            float2 s2[A][Q];
#pragma unroll
            for (int a = 0; a < A; ++a)
#pragma unroll
                for (int q = 0; q < Q; ++q) s2[a][q] = make_float2(0.f, 0.f);
#pragma unroll 2
            for (int i = 0; i < C / D; ++i) {
                const int c = i * D + d;
                float4 kx[A];
#pragma unroll
                for (int a = 0; a < A; ++a) {
                    const int key = kg + (KT / A) * a;
                    kx[a] = word(ks + key * Sh::kRow + ((c ^ swzf(key)) << 4));
                }
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const float4 qx = word(qs + (rg * Q + q) * Sh::kRow + (c << 4));
#pragma unroll
                    for (int a = 0; a < A; ++a) {
                        s2[a][q] = ffma2(make_float2(kx[a].x, kx[a].y), make_float2(qx.x, qx.y), s2[a][q]);
                        s2[a][q] = ffma2(make_float2(kx[a].z, kx[a].w), make_float2(qx.z, qx.w), s2[a][q]);
                    }
                }
            }
            float s[A * Q];
#pragma unroll
            for (int a = 0; a < A; ++a)
#pragma unroll
                for (int q = 0; q < Q; ++q) s[a * Q + q] = s2[a][q].x + s2[a][q].y;
            int first;
            lane_sums<A * Q, D>(s, lane, first);
#pragma unroll
            for (int e = 0; e < kKept<A * Q, D>; ++e) {
                const int x = first + e, a = x / Q, q = x - a * Q;
                ss[(kg + (KT / A) * a) * R + rg * Q + q] = s[e];
            }
        }
        __syncwarp();
        bool any_corr;
        {
            const int left = w.key1 - w.key0 - (w.k_first + it) * KT;
            constexpr int NK = KT > LP ? KT / LP : 1;
            float x[NK], mx = -CUDART_INF_F;
#pragma unroll
            for (int e = 0; e < NK; ++e) {
                const int key = sk + LP * e;
                x[e] = key < KT && key < left ? ss[key * R + sr] * p.scale_log2 : -CUDART_INF_F;
                mx = fmaxf(mx, x[e]);
            }
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mn = fmaxf(m_run, mx), base = mn == -CUDART_INF_F ? 0.f : mn;
            const float corr = exp2f(m_run - base);
            any_corr = __any_sync(0xffffffffu, corr != 1.f);
            m_run = mn;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < NK; ++e) {
                const int key = sk + LP * e;
                const float pe = exp2f(x[e] - base);
                sum += pe;
                if (key < KT) ss[key * R + sr] = pe;
            }
            l_run = l_run * corr + sum;  // the lane's own keys; joined at the end
            if (sk == 0) cs[sr] = corr;
        }
        __syncwarp();
        if (any_corr) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float c = cs[r];
                acc[r][0] = make_float2(acc[r][0].x * c, acc[r][0].y * c);
                acc[r][1] = make_float2(acc[r][1].x * c, acc[r][1].y * c);
            }
        }
#pragma unroll 2
        for (int key = vk; key < KT; key += VK) {
            const float4 v = word(vs + key * Sh::kRow + ((vc ^ swzf(key)) << 4));
            float pe[R];
            if constexpr (R >= 4) {
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(ss + key * R + r);
                    pe[r] = x.x;
                    pe[r + 1] = x.y;
                    pe[r + 2] = x.z;
                    pe[r + 3] = x.w;
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r) pe[r] = ss[key * R + r];
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 w2 = make_float2(pe[r], pe[r]);
                acc[r][0] = ffma2(w2, make_float2(v.x, v.y), acc[r][0]);
                acc[r][1] = ffma2(w2, make_float2(v.z, v.w), acc[r][1]);
            }
        }
        __syncwarp();  // the stage, scores and factors are read
        walk_copy<KT, Sh::kRow>(p, pl, ahead, x1, gq, words, smem_u32(ks), smem_u32(vs), swzf);
    }
    // the part
#pragma unroll
    for (int o = LP / 2; o > 0; o >>= 1) l_run += __shfl_xor_sync(0xffffffffu, l_run, o);
    const int slot = w.slot + wid;
    if (slot >= p.max_parts) return;
    if (sk == 0 && sr < w.pairs) reinterpret_cast<float2 *>(p.ws_ml)[(size_t)slot * kM + sr] = make_float2(m_run, l_run);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float4 a = make_float4(acc[r][0].x, acc[r][0].y, acc[r][1].x, acc[r][1].y);
#pragma unroll
        for (int o = 16; o >= C; o >>= 1) {  // the lanes that took other keys of the same word
            a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
            a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
            a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
            a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
        }
        if (vk == 0 && vc < words && r < w.pairs)
            reinterpret_cast<float4 *>(p.ws_acc + ((size_t)slot * kM + r) * p.head_size)[vc] = a;
    }
    __syncwarp();  // shared memory is free for the next item
}

}  // namespace

template <int HS>
__global__ void __launch_bounds__(kWalkWarps * 32, 1) attn_pages_f32_kernel(const PagesAttn p) {
    extern __shared__ __align__(128) unsigned char smem[];
    const int wid = walker_id(threadIdx.x / 32, 0);
    unsigned char *ring = smem + (threadIdx.x >> 5) * ShapeF<HS>::kWarp;
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    pdl_launch_dependents();
    if (!p.plan_in_block) pdl_wait();
    const Plan pl = plan_here<kWalkWarps * 32>(p, smem + kWalkWarps * ShapeF<HS>::kWarp, smem, blockIdx.x == 0);
    const int T_all = pl.hdr[kHdrCost], W = pl.hdr[kHdrWarps];
    const int x0 = wid < W ? first_of(wid, T_all, W) : 0, x1 = wid < W ? first_of(wid + 1, T_all, W) : 0;
    if (x0 < x1) {
        constexpr int KT = ShapeF<HS>::KT;
        int src = warp_find(&pl.src[0].t0, sizeof(Source) / 4, p.G + p.B + 1, x0), x = x0, done = 0;
        WalkAhead<KT> ahead;
        ahead.start(p, pl, src, x0, x1, gq);
        for (int s = 0; s < kStagesF; ++s) {
            const uint32_t ks = smem_u32(ring) + s * ShapeF<HS>::kStage;
            walk_copy<KT, ShapeF<HS>::kRow>(p, pl, ahead, x1, gq, p.head_size / 4, ks, ks + KT * ShapeF<HS>::kRow, swzf);
        }
        WalkItem w;
        while (walk_item(p, pl, src, x, x1, gq, w)) {
            if (w.pairs <= 1)
                walk_f32<HS, 1>(p, pl, w, ahead, x1, wid, gq, ring, done);
            else if (w.pairs <= 2)
                walk_f32<HS, 2>(p, pl, w, ahead, x1, wid, gq, ring, done);
            else if (w.pairs <= 4)
                walk_f32<HS, 4>(p, pl, w, ahead, x1, wid, gq, ring, done);
            else if (w.pairs <= 8)
                walk_f32<HS, 8>(p, pl, w, ahead, x1, wid, gq, ring, done);
            else
                walk_f32<HS, 16>(p, pl, w, ahead, x1, wid, gq, ring, done);
            done += w.n_tiles;
        }
    }
    cp_wait<0>();
}

namespace {
template <int HS>
cudaError_t launch(const PagesAttn &p, cudaLaunchConfig_t cfg) {
    auto fn = attn_pages_f32_kernel<HS>;
    static DeviceOnce once;
    cudaError_t e = once.smem(reinterpret_cast<const void *>(fn), ShapeF<HS>::kSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(p.num_sms);
    cfg.blockDim = dim3(kWalkWarps * 32);
    cfg.dynamicSmemBytes = ShapeF<HS>::kSmem;
    return cudaLaunchKernelEx(&cfg, fn, p);
}
}  // namespace

int attn_pages_f32_tile(int hs) { return hs <= 32 ? ShapeF<32>::KT : hs <= 64 ? ShapeF<64>::KT : ShapeF<128>::KT; }

cudaError_t launch_attn_pages_f32(const PagesAttn &p, cudaLaunchConfig_t cfg) {
    const int hs = p.head_size;
    return hs <= 32 ? launch<32>(p, cfg) : hs <= 64 ? launch<64>(p, cfg) : launch<128>(p, cfg);
}

}  // namespace l2
