// The paged attention over fp32 caches: one kernel whose blocks take one of two roles, the tensor-core role for shared prefixes
// (attn_pages_tc32.cuh) or the walk for everything else (see attn_pages.cu for the split into items, tiles and parts).
//
// The walk.  An item has 1 to 16 (row, head) pairs.  Up to 8, products are fp32 FMAs on the CUDA cores: a word of K or V read serves
// at most 8, 2 FMAs a byte, a third of an SM's rate when HBM feeds it.  From 9 pairs on they are mma.sync of tf32 halves,
// hi * hi + hi * lo + lo * hi (2^-21 of a product is left out); the tensor core cuts the sums it adds into, so only
// two steps of hi * hi go into one accumulator before an fp32 addition takes over, and the lo products, 2^-11 as
// large, have one of their own.  That keeps the error at that of an fp32 sum (all in one accumulator left 4 times it).
//
// FMAs.  A warp's tile is KT keys (8 KB of K and V).  Scores: a lane takes A keys by Q pairs over every D-th
// 16-byte word of the head, so each word of K read from shared memory meets Q queries and each query word A
// keys; the D lanes of a block of scores add up by a butterfly that leaves each lane its share of them.
// The scores go through shared memory once: 32 / R lanes to a pair take the softmax (running max and
// sum), then every lane holds one 16-byte word of the head for all R pairs and adds weight times V.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "../../include/l2.h"
#include "attn_pages.cuh"
#include "attn_pages_tc32.cuh"
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
    static constexpr int kS = KT * 8 * 4;         // scores, then weights [key][pair]
    static constexpr int kWarp = kStagesF * kStage + kQ + kS + kM * 4 + kItems * (int)sizeof(WalkItem);
    static constexpr int kSmem = kWalkWarps * kWarp;
};
// Head size of the tensor-core role, and the shared memory of either role, before the plan.
template <int HS>
constexpr int kTcHead = HS > 64 ? 128 : 64;
template <int HS, bool TC>
constexpr int kWorkF = TC && (int)Tc32Shape<kTcHead<HS>>::kSmem > ShapeF<HS>::kSmem ? (int)Tc32Shape<kTcHead<HS>>::kSmem : ShapeF<HS>::kSmem;

// Word c of row r sits at word c ^ swzf(r): two rows by four words, or one row by eight, fall into different banks.
__device__ __forceinline__ int swzf(int r) { return ((r & 1) << 2) | ((r >> 1) & 3); }

// How a warp's lanes divide the scores of KT keys by R pairs: D lanes along the head, A keys and all Q = R pairs a lane.
template <int KT, int R>
struct Split {
    static constexpr int D = R <= 4 || KT > 8 ? 4 : 8;
    static constexpr int Q = R;
    static constexpr int A = KT * D / 32;
    static_assert(A >= 1 && (KT / A) * D == 32, "the lanes must cover the scores once");
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

// A warp's state for its item: running sums of word vc of the head for up to 8 pairs, over keys vk, vk + VK, .. of each tile;
// softmax state of the pair this lane serves.
template <int HS>
struct StateF {
    float2 acc[HS / 8 > 8 ? HS / 8 : 8][2];
    float m, l;
};

// One tile of an item of at most R pairs: left keys from its first on.
template <int HS, int R>
__device__ __forceinline__ void tile_f32(StateF<HS> &st, const unsigned char *ks, const unsigned char *qs, float *ss, float *cs, int left,
                                         float scale_log2) {
    using Sh = ShapeF<HS>;
    constexpr int KT = Sh::KT, C = Sh::C;
    using Sp = Split<KT, R>;
    constexpr int A = Sp::A, Q = Sp::Q, D = Sp::D;
    const int lane = threadIdx.x & 31;
    const unsigned char *vs = ks + KT * Sh::kRow;
    auto word = [](const unsigned char *a) { return *reinterpret_cast<const float4 *>(a); };
    // scores: D lanes along the head, then keys
    const int d = lane % D, kg = lane / D;
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
                const float4 qx = word(qs + q * Sh::kRow + (c << 4));
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
            ss[(kg + (KT / A) * a) * R + q] = s[e];
        }
    }
    __syncwarp();
    // softmax: LP lanes to pair sr
    constexpr int LP = 32 / R, NK = KT > LP ? KT / LP : 1;
    const int sr = lane / LP, sk = lane % LP;
    float x[NK], mx = -CUDART_INF_F;
#pragma unroll
    for (int e = 0; e < NK; ++e) {
        const int key = sk + LP * e;
        x[e] = key < KT && key < left ? ss[key * R + sr] * scale_log2 : -CUDART_INF_F;
        mx = fmaxf(mx, x[e]);
    }
#pragma unroll
    for (int o = LP / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(st.m, mx), base = mn == -CUDART_INF_F ? 0.f : mn;
    const float corr = exp2f(st.m - base);
    st.m = mn;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < NK; ++e) {
        const int key = sk + LP * e;
        const float pe = exp2f(x[e] - base);
        sum += pe;
        if (key < KT) ss[key * R + sr] = pe;
    }
    st.l = st.l * corr + sum;  // the lane's own keys; joined at the end
    if (sk == 0) cs[sr] = corr;
    __syncwarp();
    // the tile's sums by themselves, so that a long walk is a chain of tiles and not of keys: 20000 keys a warp, error 5.7e-7 in
    // place of 1.6e-6 (torch's fp32 products: 4.9e-7), for 3 % at 8 pairs
    float2 t[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) t[r][0] = t[r][1] = make_float2(0.f, 0.f);
    constexpr int VK = 32 / C;
    const int vc = lane % C, vk = lane / C;
#pragma unroll 2
    for (int key = vk; key < KT; key += VK) {
        const float4 v = word(vs + key * Sh::kRow + ((vc ^ swzf(key)) << 4));
        float pe[R];
        if constexpr (R >= 4) {
#pragma unroll
            for (int r = 0; r < R; r += 4) {
                const float4 y = *reinterpret_cast<const float4 *>(ss + key * R + r);
                pe[r] = y.x;
                pe[r + 1] = y.y;
                pe[r + 2] = y.z;
                pe[r + 3] = y.w;
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) pe[r] = ss[key * R + r];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 w2 = make_float2(pe[r], pe[r]);
            t[r][0] = ffma2(w2, make_float2(v.x, v.y), t[r][0]);
            t[r][1] = ffma2(w2, make_float2(v.z, v.w), t[r][1]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float2 c = make_float2(cs[r], cs[r]);
        st.acc[r][0] = ffma2(st.acc[r][0], c, t[r][0]);
        st.acc[r][1] = ffma2(st.acc[r][1], c, t[r][1]);
    }
}

// D = A B of m16n8k8 in tf32 (add: + D).
__device__ __forceinline__ void mma_tf32_to(float *d, const uint32_t *a, uint32_t b0, uint32_t b1, bool add) {
    const float z = 0.f;
    if (add)
        asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z));
}
// x = hi + lo in tf32, to 2^-22 of x
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}
// The same for a value that stays in the output: hi is at most tf32's largest, so that a finite x does not round to infinity (but for the
// two largest floats, whose halves add up to 2^128).  An infinite or NaN x is one in lo.
__device__ __forceinline__ void split_tf32_finite(float x, uint32_t &hi, uint32_t &lo) {
    float y;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(__uint_as_float(0x7f7fe000u)));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(y));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}
// Columns 2 t4 + e of n8 tile 4 i + j of the sums are dimensions 32 i + 4 w(2 t4 + e) + j: the word of V a lane reads, chosen
// so that a phase's eight reads fall into different banks.
__device__ __forceinline__ int v_word(int g) { return ((g & 1) << 2) | (g >> 1); }

// One tile of an item of more than 8 pairs, which are the rows of the products.  The sums of rows g4 and g4 + 8 live in
// st.acc as n8 tiles; m2, l2: their softmax state.
template <int HS>
__device__ __forceinline__ void tile_mma(StateF<HS> &st, float *m2, float *l2, const unsigned char *ks, const unsigned char *qs, int left,
                                         float scale_log2) {
    using Sh = ShapeF<HS>;
    constexpr int KT = Sh::KT, NT = KT / 8;
    const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
    const unsigned char *vs = ks + KT * Sh::kRow;
    auto word = [](const unsigned char *a) { return *reinterpret_cast<const float4 *>(a); };
    float s[NT][4], sl[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][j] = sl[n][j] = 0.f;
    // K steps 2 i and 2 i + 1 of 8 take dimensions 16 i + 4 t4 + {0, 1} and {2, 3}: one 16-byte read a row
#pragma unroll 2
    for (int i = 0; i < HS / 16; ++i) {
        const float4 a = word(qs + g4 * Sh::kRow + 64 * i + 16 * t4), b = word(qs + (g4 + 8) * Sh::kRow + 64 * i + 16 * t4);
        uint32_t qh[8], ql[8];
        split_tf32(a.x, qh[0], ql[0]);
        split_tf32(b.x, qh[1], ql[1]);
        split_tf32(a.y, qh[2], ql[2]);
        split_tf32(b.y, qh[3], ql[3]);
        split_tf32(a.z, qh[4], ql[4]);
        split_tf32(b.z, qh[5], ql[5]);
        split_tf32(a.w, qh[6], ql[6]);
        split_tf32(b.w, qh[7], ql[7]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int key = 8 * n + g4;
            const float4 x = word(ks + key * Sh::kRow + (((4 * i + t4) ^ swzf(key)) << 4));
            uint32_t h[4], l[4];
            split_tf32(x.x, h[0], l[0]);
            split_tf32(x.y, h[1], l[1]);
            split_tf32(x.z, h[2], l[2]);
            split_tf32(x.w, h[3], l[3]);
            float c[4];
            mma_tf32_to(c, qh, h[0], h[1], false);
            mma_tf32_to(c, qh + 4, h[2], h[3], true);
            mma_tf32_to(sl[n], ql, h[0], h[1], true);
            mma_tf32_to(sl[n], ql + 4, h[2], h[3], true);
            mma_tf32_to(sl[n], qh, l[0], l[1], true);
            mma_tf32_to(sl[n], qh + 4, l[2], l[3], true);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[n][j] += c[j];
        }
    }
    bool odd = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[n][j] += sl[n][j];
            odd |= s[n][j] != s[n][j];
        }
    // the halves of an infinity make NaN of a score that may be infinite: such tiles are summed again as they are
    if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = 8 * n + 2 * t4 + (j & 1), row = g4 + 8 * (j >> 1);
                s[n][j] = 0.f;
#pragma unroll 1
                for (int c = 0; c < Sh::C; ++c) {
                    const float4 x = word(ks + key * Sh::kRow + ((c ^ swzf(key)) << 4)), y = word(qs + row * Sh::kRow + (c << 4));
                    s[n][j] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[n][j]))));
                }
            }
    }
    float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = 8 * n + 2 * t4 + (j & 1);
            s[n][j] = key < left ? s[n][j] * scale_log2 : -CUDART_INF_F;
            mx[j >> 1] = fmaxf(mx[j >> 1], s[n][j]);
        }
    float corr[2], base[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        const float mn = fmaxf(m2[r], mx[r]);
        base[r] = mn == -CUDART_INF_F ? 0.f : mn;
        corr[r] = exp2f(m2[r] - base[r]);
        m2[r] = mn;
        l2[r] *= corr[r];
    }
    uint32_t ph[NT][4], plo[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[n][j] = exp2f(s[n][j] - base[j >> 1]);
            l2[j >> 1] += s[n][j];
        }
        // key slots t4 and t4 + 4 of a step are keys 2 t4 and 2 t4 + 1: the weights are A fragments as they come
        split_tf32(s[n][0], ph[n][0], plo[n][0]);
        split_tf32(s[n][2], ph[n][1], plo[n][1]);
        split_tf32(s[n][1], ph[n][2], plo[n][2]);
        split_tf32(s[n][3], ph[n][3], plo[n][3]);
    }
    const int vw = v_word(g4);
#pragma unroll
    for (int i = 0; i < HS / 32; ++i) {
        float acc[4][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int key = 8 * n + 2 * t4;
            const float4 x0 = word(vs + key * Sh::kRow + (((8 * i + vw) ^ swzf(key)) << 4));
            const float4 x1 = word(vs + (key + 1) * Sh::kRow + (((8 * i + vw) ^ swzf(key + 1)) << 4));
            const float a0[4] = {x0.x, x0.y, x0.z, x0.w}, a1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t h0, l0, h1, l1;
                split_tf32_finite(a0[j], h0, l0);
                split_tf32_finite(a1[j], h1, l1);
                mma_tf32_to(acc[j], plo[n], h0, h1, n > 0);
                mma_tf32_to(acc[j], ph[n], l0, l1, true);
                mma_tf32_to(acc[j], ph[n], h0, h1, true);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 *o = st.acc[(4 * i + j)];
            o[0] = make_float2(fmaf(o[0].x, corr[0], acc[j][0]), fmaf(o[0].y, corr[0], acc[j][1]));
            o[1] = make_float2(fmaf(o[1].x, corr[1], acc[j][2]), fmaf(o[1].y, corr[1], acc[j][3]));
        }
    }
}

// The walk of one warp: number `warp` of its block's, whose first walking one is block0.
template <int HS>
__device__ __forceinline__ void walk_f32(const PagesAttn &p, const Plan &pl, unsigned char *smem, int warp, int block0) {
    using Sh = ShapeF<HS>;
    constexpr int KT = Sh::KT, C = Sh::C;
    const int lane = threadIdx.x & 31, wid = walker_id(warp, block0);
    unsigned char *ring = smem + warp * Sh::kWarp, *qs = ring + kStagesF * Sh::kStage;
    float *ss = reinterpret_cast<float *>(qs + Sh::kQ), *cs = ss + Sh::kS / 4;
    WalkItem *queue = reinterpret_cast<WalkItem *>(cs + kM);
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads), words = p.head_size / 4;
    Walk<KT, Sh::kRow> walk;
    walk.start(pl, wid, p.G + p.B);
    StateF<HS> st;
    float m2[2], l2[2];
    WalkItem w = {};
    int it = 0, items = 0;  // tile within the item, items taken
    // step s copies tile s - 1 and computes tile s - kStagesF
#pragma unroll 1
    for (int step = 0;; ++step) {
        {
            const uint32_t to = smem_u32(ring) + ((step + kStagesF - 1) % kStagesF) * Sh::kStage;
            walk.step(p, pl, gq, words, queue, to, to + KT * Sh::kRow, swzf);
        }
        if (step < kStagesF) continue;
        if (step - kStagesF >= walk.issued) break;
        if (it == 0) {
            __syncwarp();  // the item was written by lane 0
            w = queue[items++ % kItems];
            const int n = w.pairs <= 8 ? 8 : kM;
#pragma unroll 1
            for (int e = lane; e < n * C; e += 32) {
                const int i = e / C, c = e % C;
                const char *q = walk_query(p, w, i, gq);
                *reinterpret_cast<float4 *>(qs + i * Sh::kRow + (c << 4)) =
                    q && c < words ? reinterpret_cast<const float4 *>(q)[c] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            st.m = -CUDART_INF_F;
            st.l = 0.f;
            m2[0] = m2[1] = -CUDART_INF_F;
            l2[0] = l2[1] = 0.f;
#pragma unroll
            for (int r = 0; r < (HS / 8 > 8 ? HS / 8 : 8); ++r) st.acc[r][0] = st.acc[r][1] = make_float2(0.f, 0.f);
        }
        cp_wait<kStagesF - 1>();
        __syncwarp();
        const unsigned char *ks = ring + (step % kStagesF) * Sh::kStage;
        const int left = w.left - it * KT;
        if (w.pairs <= 1)
            tile_f32<HS, 1>(st, ks, qs, ss, cs, left, p.scale_log2);
        else if (w.pairs <= 2)
            tile_f32<HS, 2>(st, ks, qs, ss, cs, left, p.scale_log2);
        else if (w.pairs <= 4)
            tile_f32<HS, 4>(st, ks, qs, ss, cs, left, p.scale_log2);
        else if (w.pairs <= 8)
            tile_f32<HS, 8>(st, ks, qs, ss, cs, left, p.scale_log2);
        else
            tile_mma<HS>(st, m2, l2, ks, qs, left, p.scale_log2);
        if (++it == w.n_tiles) {
            // the part
            it = 0;
            const int slot = w.slot + wid;
            float2 *ml = reinterpret_cast<float2 *>(p.ws_ml) + (size_t)slot * kM;
            float *to = p.ws_acc + (size_t)slot * kM * p.head_size;
            if (slot >= p.max_parts) {
            } else if (w.pairs <= 8) {
                const int R = w.pairs <= 1 ? 1 : w.pairs <= 2 ? 2 : w.pairs <= 4 ? 4 : 8, LP = 32 / R;
                const int sr = lane / LP, vc = lane % C, vk = lane / C;
                for (int o = LP / 2; o > 0; o >>= 1) st.l += __shfl_xor_sync(0xffffffffu, st.l, o);
                if (lane % LP == 0 && sr < w.pairs) ml[sr] = make_float2(st.m, st.l);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if (r >= w.pairs) continue;
                    float4 a = make_float4(st.acc[r][0].x, st.acc[r][0].y, st.acc[r][1].x, st.acc[r][1].y);
#pragma unroll
                    for (int o = 16; o >= C; o >>= 1) {  // the lanes that took other keys of the same word
                        a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
                        a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
                        a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
                        a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
                    }
                    if (vk == 0 && vc < words) reinterpret_cast<float4 *>(to + r * p.head_size)[vc] = a;
                }
            } else {
                const int g4 = lane >> 2, t4 = lane & 3;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float l = l2[r];
                    l += __shfl_xor_sync(0xffffffffu, l, 1);
                    l += __shfl_xor_sync(0xffffffffu, l, 2);
                    const int pr = g4 + 8 * r;
                    if (pr >= w.pairs) continue;
                    if (t4 == 0) ml[pr] = make_float2(m2[r], l);
#pragma unroll
                    for (int i = 0; i < HS / 32; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int c = 8 * i + v_word(2 * t4 + e);
                            auto at = [&](int j) { return e ? st.acc[4 * i + j][r].y : st.acc[4 * i + j][r].x; };
                            if (c < words) reinterpret_cast<float4 *>(to + pr * p.head_size)[c] = make_float4(at(0), at(1), at(2), at(3));
                        }
                }
            }
        }
        __syncwarp();  // the stage, scores and factors are read before they are written again
    }
    cp_wait<0>();
}

}  // namespace

// TC: blocks below the plan's share take the tensor-core role, the others walk.  Calls that have no use for it have a kernel of
// the walk alone, of fewer threads, which is up sooner.
template <int HS, bool TC>
__global__ void __launch_bounds__(attn_threads(TC), 1) attn_pages_f32_kernel(const __grid_constant__ PagesAttn p) {
    extern __shared__ __align__(1024) unsigned char smem[];
    pdl_launch_dependents();
    pdl_wait();
    const Plan pl = plan_here<attn_threads(TC)>(p, smem + kWorkF<HS, TC>, smem, blockIdx.x == 0);
    const int n_tc = TC ? pl.hdr[kHdrTcBlocks] : 0, warp = threadIdx.x / 32 - walk_first(TC);
    if constexpr (TC) {
        if ((int)blockIdx.x < n_tc) return tc32_role<kTcHead<HS>>(p, pl, smem, blockIdx.x);
        // the four warps that do not walk leave their registers to the eight that do: 24 + 2 * 240 = 3 * 168
        if (warp < 0) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 24;");
            return;
        }
        asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
    }
    walk_f32<HS>(p, pl, smem, warp, n_tc);
}

namespace {
template <int HS, bool TC>
cudaError_t launch(const PagesAttn &p, cudaLaunchConfig_t cfg) {
    constexpr int bytes = kWorkF<HS, TC> + (int)kPlanSmem;
    auto fn = attn_pages_f32_kernel<HS, TC>;
    static DeviceOnce once;
    cudaError_t e = once.smem(reinterpret_cast<const void *>(fn), bytes, TC ? 168 : 0);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(p.num_sms);
    cfg.blockDim = dim3(attn_threads(TC));
    cfg.dynamicSmemBytes = bytes;
    return cudaLaunchKernelEx(&cfg, fn, p);
}
template <int HS>
cudaError_t launch(const PagesAttn &p, cudaLaunchConfig_t cfg) {
    return p.tc ? launch<HS, true>(p, cfg) : launch<HS, false>(p, cfg);
}
}  // namespace

int attn_pages_f32_shift(int hs) { return hs <= 32 ? 5 : hs <= 64 ? 4 : 3; }
static_assert(ShapeF<32>::KT == 1 << 5 && ShapeF<64>::KT == 1 << 4 && ShapeF<128>::KT == 1 << 3, "the plan counts tiles by shifts");

cudaError_t launch_attn_pages_f32(const PagesAttn &p, cudaLaunchConfig_t cfg) {
    const int hs = p.head_size;
    return hs <= 32 ? launch<32>(p, cfg) : hs <= 64 ? launch<64>(p, cfg) : launch<128>(p, cfg);
}

}  // namespace l2
