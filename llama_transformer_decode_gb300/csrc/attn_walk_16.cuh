// The paged attention over 16-bit caches: one kernel whose blocks take one of two roles, the tensor-core role for shared
// prefixes (attn_pages_tc.cuh) or the walk for everything else (see attn_pages.cu for the split into items, tiles and parts).
// The plan divides the blocks by the roles' costs, so the two run side by side, with one launch and one start-up.
//
// The walk.  A warp's 16 pairs are the M of mma.sync m16n8k16 against its tile's keys (16 products per word read: reading
// bounds it, at 5.8 to 6.2 TB/s of suffixes of 4000 rows, and a warp needs no other); q, K and V as
// stored, and the weights 2^(x - m) as a sum of two 16-bit values, so nothing is rounded but the fp32 sums and the output.
// Eight warps of a block walk, each with three tiles (24 KB) of its own.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "../../include/l2.h"
#include "attn_pages.cuh"
#include "attn_pages_tc.cuh"
#include "attn_plan.cuh"
#include "l2_device.cuh"
#include "l2_pages.h"

namespace l2 {

namespace {

constexpr int kStages = 3;                      // tiles of a warp's ring

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

// kLift: the weights of a tile are 2^(x - max + kLift).  In fp16, whose least step is 2^-24, weights far below the
// largest would otherwise be lost, and there may be 10^5 of them; in bf16 the exponent is that of fp32.
struct TBf16 {
    static constexpr float kLift = 0.f;
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
    static constexpr uint32_t kExponent = 0x7f807f80u;  // all ones in infinities and NaN
};
struct TF16 {
    static constexpr float kLift = 15.f;
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
    static constexpr uint32_t kExponent = 0x7c007c00u;
};
// All ones in the halves of v that are infinite or NaN.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t v) {
    return __vcmpeq2(v & T::kExponent, T::kExponent);
}

// Tile shape: HS the head size padded to 64 or 128; K and V of a tile's keys take 8 KB, or of a team's 16 KB where heads are 128.  A team
// has its warps' shared memory together, so more stages.
template <int HS, int TEAM>
struct Shape {
    static constexpr int KT = HS == 128 && TEAM == 1 ? 16 : 32;
    static constexpr int C = HS * 2 / 16;         // 16-byte words a row
    static constexpr int kRow = HS * 2;
    static constexpr int kStage = 2 * KT * kRow;  // K then V
    static constexpr int kWarps = walk_warps(false, TEAM), kTeams = kWarps / TEAM;
    static constexpr int kRings = kWalkWarps * kStages * 8192;
    static constexpr int kDepth = kRings / kTeams / kStage;  // stages of a ring
    static_assert(kDepth >= 2 && kDepth * kTeams * kStage <= kRings, "the rings' memory");
    static constexpr int kItems = ring_items(TEAM);
    static constexpr int kSmem = kRings + kWarps * kItems * (int)sizeof(WalkItem);
    static_assert(kDepth < kItems, "a walk's ring of items");
};
// Shared memory of either role, before the plan.
template <int HS, bool TC, int TEAM>
constexpr int kWork = TC && (int)TcShape<HS>::kSmem > Shape<HS, TEAM>::kSmem ? (int)TcShape<HS>::kSmem : Shape<HS, TEAM>::kSmem;

// Threads of a block: teams take all of its warps, with the tensor-core role or without.
__host__ __device__ constexpr int walk_threads(bool tc, int team) { return team == 1 ? attn_threads(tc) : 32 * kTeamWarps; }
static_assert(32 * kTeamWarps == attn_threads(true), "the tensor-core role has as many warps");

// Word c of row r sits at word c ^ swz(r): the eight rows that one ldmatrix phase reads fall into
// different banks.
__device__ __forceinline__ int swz(int r) { return r & 7; }

// The walk of one warp (see the head of attn_pages.cu): number `warp` of its block's, whose first walking one is block0.
// TREE: the rows are drafted tokens, and of the sequence's last keys a row sees its own path (see tree_bits).  What a row does not
// see has no weight, but 0 times an infinity or NaN of V is NaN: tiles with drafted keys are looked through for such values, which then
// stay out of the product and are added one by one to the rows that see them.
// TEAM > 1: so many warps are one walker, with a ring together and 16 pairs each.  Where a sequence has more pairs than 16, each warp for itself
// would bring the keys in anew (32 sequences of 8000 keys, 8 KV heads of 128: 173 us with 16 pairs, 323 with 32, 628 with 64;
// teams of two and four take 217 and 388).
template <typename T, int HS, bool TREE, int TEAM>
__device__ __forceinline__ void walk_role(const PagesAttn &p, const Plan &pl, unsigned char *smem, int warp, int block0) {
    using Sh = Shape<HS, TEAM>;
    constexpr int KT = Sh::KT, C = Sh::C, NT = KT / 8;  // NT: n8 tiles of keys
    constexpr int kStages = Sh::kDepth;
    const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3, team = warp / TEAM, member = warp % TEAM, wid = walker_id(team, block0);
    const uint32_t ring = smem_u32(smem) + team * (kStages * Sh::kStage);
    WalkItem *queue = reinterpret_cast<WalkItem *>(smem + Sh::kRings) + warp * Sh::kItems;
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    const int words = p.head_size / 8;  // 16-byte words of a row that exist
    Walk<KT, Sh::kRow, TREE, TEAM> walk;
    walk.start(p, pl, wid);
    float m_run[2], l_run[2], o[HS / 8][4];
    constexpr int QR = HS / 16 * 4;
    uint32_t qf[QR];
    WalkItem w = {};
    TreeItem tree = {};
    int it = 0, items = 0;  // tile within the item, items taken
    // step s copies tile s - 1 and computes tile s - kStages
#pragma unroll 1
    for (int step = 0;; ++step) {
        if constexpr (TEAM > 1)
            if (step >= kStages) {
                // the next tile is here, and all of the team are done with the one whose stage is copied into
                cp_wait<kStages - 2>();
                team_sync<TEAM>(team);
            }
        {
            const uint32_t st = ring + ((step + kStages - 1) % kStages) * Sh::kStage;
            walk.step(p, pl, gq, words, queue, st, st + KT * Sh::kRow, swz, member);
        }
        if (step < kStages) continue;
        if (step - kStages >= walk.issued) break;
        if (it == 0) {
            __syncwarp();  // the item was written by lane 0
            w = queue[items++ % Sh::kItems];
            if constexpr (TREE) tree = tree_item<KT>(p, w, gq, member);
            const char *qa = walk_query(p, w, g4, gq), *qb = walk_query(p, w, g4 + 8, gq);
            m_run[0] = m_run[1] = -CUDART_INF_F;
            l_run[0] = l_run[1] = 0.f;
#pragma unroll
            for (int i = 0; i < HS / 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
            // The A fragments of all K steps: word t4 of every 16-byte chunk of rows g4 and g4 + 8.  Each lane loads every fourth
            // chunk whole (few loads, all in flight) and the four lanes of a row exchange words.
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 *q4 = reinterpret_cast<const uint4 *>(r ? qb : qa);
                uint4 v[HS / 32];
#pragma unroll
                for (int i = 0; i < HS / 32; ++i) v[i] = q4 && 4 * i + t4 < words ? q4[4 * i + t4] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int i = 0; i < HS / 32; ++i) {
                    // 4 x 4 transpose: lane t4 ends with word t4 of chunks 4 i .. 4 i + 3
                    const bool o1 = t4 & 1, o2 = t4 & 2;
                    uint32_t a0 = __shfl_xor_sync(0xffffffffu, o1 ? v[i].x : v[i].y, 1), a1 = __shfl_xor_sync(0xffffffffu, o1 ? v[i].z : v[i].w, 1);
                    const uint32_t x0 = o1 ? a0 : v[i].x, x1 = o1 ? v[i].y : a0, x2 = o1 ? a1 : v[i].z, x3 = o1 ? v[i].w : a1;
                    a0 = __shfl_xor_sync(0xffffffffu, o2 ? x0 : x2, 2);
                    a1 = __shfl_xor_sync(0xffffffffu, o2 ? x1 : x3, 2);
                    // chunk 4 i + c is half c & 1 of K step 2 i + c / 2
                    qf[8 * i + r] = o2 ? a0 : x0;
                    qf[8 * i + 2 + r] = o2 ? a1 : x1;
                    qf[8 * i + 4 + r] = o2 ? x2 : a0;
                    qf[8 * i + 6 + r] = o2 ? x3 : a1;
                }
            }
        }
        if constexpr (TEAM == 1) {
            cp_wait<kStages - 1>();
            __syncwarp();
        }
        const uint32_t ks_base = ring + (step % kStages) * Sh::kStage, vs_base = ks_base + KT * Sh::kRow;
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

        // scale, mask keys past the end and those not seen, running max
        const int left = w.left - it * KT;
        const bool drafted = TREE && left - KT < tree.n;  // the tile reaches drafted keys
        unsigned sees[2] = {~0u, ~0u};
        bool odd = false;  // V has infinities or NaN
        if constexpr (TREE)
            if (drafted) {
                const unsigned mine = tree_bits(tree.sees, tree.n, left);
                sees[0] = __shfl_sync(0xffffffffu, mine, g4);
                sees[1] = __shfl_sync(0xffffffffu, mine, g4 + 8);
                const uint4 *vt = reinterpret_cast<const uint4 *>(smem + (vs_base - smem_u32(smem)));
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < KT * C / 32; ++i) {
                    const uint4 x = vt[i * 32 + lane];
                    any |= not_finite<T>(x.x) | not_finite<T>(x.y) | not_finite<T>(x.z) | not_finite<T>(x.w);
                }
                odd = __any_sync(0xffffffffu, any != 0);
            }
        float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = 8 * n + 2 * t4 + (j & 1);
                const bool on = key < left && (!TREE || (sees[j >> 1] >> key & 1));
                s[n][j] = on ? s[n][j] * p.scale_log2 : -CUDART_INF_F;
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
            base[r] -= T::kLift;
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
        if constexpr (TREE)
            if (odd) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll 1
                    for (int kk = 0; kk < 8; ++kk) {
                        // the weights of key 8 n + kk in rows g4 and g4 + 8 are in lane kk / 2 of the four that share them
                        const int key = 8 * n + kk, from = (lane & ~3) | kk >> 1;
                        const float wa = __shfl_sync(0xffffffffu, kk & 1 ? s[n][1] : s[n][0], from);
                        const float wb = __shfl_sync(0xffffffffu, kk & 1 ? s[n][3] : s[n][2], from);
                        const unsigned char *row = smem + (vs_base - smem_u32(smem)) + key * Sh::kRow + 4 * t4;
#pragma unroll
                        for (int i = 0; i < HS / 8; ++i) {
                            const uint32_t x = *reinterpret_cast<const uint32_t *>(row + ((i ^ swz(key)) << 4)), bad = not_finite<T>(x);
                            const float2 v = T::unpack(x);
                            if ((bad & 0xffffu) && (sees[0] >> key & 1)) o[i][0] = fmaf(wa, v.x, o[i][0]);
                            if ((bad >> 16) && (sees[0] >> key & 1)) o[i][1] = fmaf(wa, v.y, o[i][1]);
                            if ((bad & 0xffffu) && (sees[1] >> key & 1)) o[i][2] = fmaf(wb, v.x, o[i][2]);
                            if ((bad >> 16) && (sees[1] >> key & 1)) o[i][3] = fmaf(wb, v.y, o[i][3]);
                        }
                    }
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
                if (TREE && odd) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] &= ~not_finite<T>(b[j]);
                }
                T::mma(o[c], ph, b[0], b[1]);
                T::mma(o[c], plo, b[0], b[1]);
                T::mma(o[c + 1], ph, b[2], b[3]);
                T::mma(o[c + 1], plo, b[2], b[3]);
            }
        }
        if (++it == w.n_tiles) {
            it = 0;
            // the part: (m, l) and the sums of the item's pairs
            const int slot = w.slot + wid;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = l_run[r];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                const int mi = g4 + 8 * r;
                if (mi >= w.pairs || slot >= p.max_parts) continue;
                const size_t at = (size_t)slot * (kM * TEAM) + kM * member + mi;
                if (t4 == 0) reinterpret_cast<float2 *>(p.ws_ml)[at] = make_float2(m_run[r] - T::kLift, l);
                float *dst = p.ws_acc + at * p.head_size;
#pragma unroll
                for (int i = 0; i < HS / 8; ++i) {
                    const int d = 8 * i + 2 * t4;
                    if (d < p.head_size) *reinterpret_cast<float2 *>(dst + d) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
                }
            }
        }
        if constexpr (TEAM == 1) __syncwarp();  // the stage is read before the next copy into it
    }
    cp_wait<0>();
}

}  // namespace

// TC: blocks below the plan's share take the tensor-core role, the others walk.  Calls that have no use for it have a kernel of
// the walk alone, of fewer threads, which is up sooner.
template <typename T, int HS, bool BF, bool TC, bool TREE, int TEAM>
__global__ void __launch_bounds__(walk_threads(TC, TEAM), 1) attn_pages_16_kernel(const __grid_constant__ TcAttn ta) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const PagesAttn &p = ta.p;
    pdl_launch_dependents();
    pdl_wait();
    const Plan pl = plan_here<walk_threads(TC, TEAM), TREE>(p, smem + kWork<HS, TC, TEAM>, smem, blockIdx.x == 0);
    const int n_tc = TC ? pl.hdr[kHdrTcBlocks] : 0, warp = threadIdx.x / 32 - (TEAM == 1 ? walk_first(TC) : 0);
    if constexpr (TC) {
        if ((int)blockIdx.x < n_tc) return tc_role<HS, BF>(ta, pl, smem, blockIdx.x);
        if constexpr (TEAM == 1) {
            // the four warps that do not walk leave their registers to the eight that do: 24 + 2 * 240 = 3 * 168
            if (warp < 0) {
                asm volatile("setmaxnreg.dec.sync.aligned.u32 24;");
                return;
            }
            asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
        }
    }
    walk_role<T, HS, TREE, TEAM>(p, pl, smem, warp, n_tc);
}

namespace {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

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

template <typename T, int HS, bool BF, bool TC, bool TREE, int TEAM>
cudaError_t launch(const TcAttn &ta, cudaLaunchConfig_t cfg) {
    constexpr int bytes = kWork<HS, TC, TEAM> + (int)kPlanSmem;
    auto fn = attn_pages_16_kernel<T, HS, BF, TC, TREE, TEAM>;
    static DeviceOnce once;
    cudaError_t e = once.smem(reinterpret_cast<const void *>(fn), bytes, TC && TEAM == 1 ? 168 : 0);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(ta.p.num_sms);
    cfg.blockDim = dim3(walk_threads(TC, TEAM));
    cfg.dynamicSmemBytes = bytes;
    return cudaLaunchKernelEx(&cfg, fn, ta);
}
template <typename T, int HS, bool BF, bool TREE>
cudaError_t launch(const TcAttn &ta, cudaLaunchConfig_t cfg) {
    if constexpr (TREE) {
        if (ta.p.team == 4) return ta.p.tc ? launch<T, HS, BF, true, true, 4>(ta, cfg) : launch<T, HS, BF, false, true, 4>(ta, cfg);
        if (ta.p.team == 2) return ta.p.tc ? launch<T, HS, BF, true, true, 2>(ta, cfg) : launch<T, HS, BF, false, true, 2>(ta, cfg);
    }
    return ta.p.tc ? launch<T, HS, BF, true, TREE, 1>(ta, cfg) : launch<T, HS, BF, false, TREE, 1>(ta, cfg);
}

template <bool TREE>
cudaError_t launch_16(const PagesAttn &p, cudaLaunchConfig_t cfg) {
    TcAttn ta{};
    ta.p = p;
    ta.box_rows = p.page_size < tc_keys(false) ? p.page_size : tc_keys(false);
    ta.scale_log2 = p.scale_log2 < 0.f ? -p.scale_log2 : p.scale_log2;
    ta.flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    if (p.tc && (!encode_pages(&ta.kmap, p.k, p, ta.box_rows) || !encode_pages(&ta.vmap, p.v, p, ta.box_rows))) return cudaErrorInvalidValue;
    if (p.head_size <= 64) return p.dtype == L2_BF16 ? launch<TBf16, 64, true, TREE>(ta, cfg) : launch<TF16, 64, false, TREE>(ta, cfg);
    return p.dtype == L2_BF16 ? launch<TBf16, 128, true, TREE>(ta, cfg) : launch<TF16, 128, false, TREE>(ta, cfg);
}

}  // namespace

}  // namespace l2
