// The paged attention over 16-bit caches: one kernel whose blocks take one of two roles, the tensor-core role for shared
// prefixes (attn_pages_tc.cuh) or the walk for everything else (see attn_pages.cu for the split into items, tiles and parts).
// The plan divides the blocks by the roles' costs, so the two run side by side, with one launch and one start-up.
//
// The walk.  A warp's 16 pairs are the M of mma.sync m16n8k16 against its tile's keys (16 products per word read: reading
// bounds it, at 5.8 to 6.2 TB/s of suffixes of 4000 rows, and a warp needs no other); q, K and V as
// stored, and the weights 2^(x - m) as a sum of two 16-bit values, so nothing is rounded but the fp32 sums and the output.
// Eight warps of a block walk, each with three tiles (24 KB) of its own.
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
};

// Tile shape: HS the head size padded to 64 or 128; K and V of a tile's keys take 8 KB.
template <int HS>
struct Shape {
    static constexpr int KT = HS == 128 ? 16 : 32;
    static constexpr int C = HS * 2 / 16;         // 16-byte words a row
    static constexpr int kRow = HS * 2;
    static constexpr int kStage = 2 * KT * kRow;  // K then V
    static constexpr int kRings = kWalkWarps * kStages * kStage;
    static constexpr int kSmem = kRings + kWalkWarps * kItems * (int)sizeof(WalkItem);
};
// Shared memory of either role, before the plan.
template <int HS, bool TC>
constexpr int kWork = TC && (int)TcShape<HS>::kSmem > Shape<HS>::kSmem ? (int)TcShape<HS>::kSmem : Shape<HS>::kSmem;

// Word c of row r sits at word c ^ swz(r): the eight rows that one ldmatrix phase reads fall into
// different banks.
__device__ __forceinline__ int swz(int r) { return r & 7; }

// The walk of one warp (see the head of attn_pages.cu): number `warp` of its block's, whose first walking one is block0.
template <typename T, int HS>
__device__ __forceinline__ void walk_role(const PagesAttn &p, const Plan &pl, unsigned char *smem, int warp, int block0) {
    using Sh = Shape<HS>;
    constexpr int KT = Sh::KT, C = Sh::C, NT = KT / 8;  // NT: n8 tiles of keys
    const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3, wid = walker_id(warp, block0);
    const uint32_t ring = smem_u32(smem) + warp * (kStages * Sh::kStage);
    WalkItem *queue = reinterpret_cast<WalkItem *>(smem + Sh::kRings) + warp * kItems;
    const int gq = heads_per_kv(p.n_heads, p.n_kv_heads);
    const int words = p.head_size / 8;  // 16-byte words of a row that exist
    Walk<KT, Sh::kRow> walk;
    walk.start(pl, wid, p.G + p.B);
    float m_run[2], l_run[2], o[HS / 8][4];
    constexpr int QR = HS / 16 * 4;
    uint32_t qf[QR];
    WalkItem w = {};
    int it = 0, items = 0;  // tile within the item, items taken
    // step s copies tile s - 1 and computes tile s - kStages
#pragma unroll 1
    for (int step = 0;; ++step) {
        {
            const uint32_t st = ring + ((step + kStages - 1) % kStages) * Sh::kStage;
            walk.step(p, pl, gq, words, queue, st, st + KT * Sh::kRow, swz);
        }
        if (step < kStages) continue;
        if (step - kStages >= walk.issued) break;
        if (it == 0) {
            __syncwarp();  // the item was written by lane 0
            w = queue[items++ % kItems];
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
        cp_wait<kStages - 1>();
        __syncwarp();
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

        // scale, mask keys past the end, running max
        const int left = w.left - it * KT;
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
                if (t4 == 0) reinterpret_cast<float2 *>(p.ws_ml)[(size_t)slot * kM + mi] = make_float2(m_run[r] - T::kLift, l);
                float *dst = p.ws_acc + ((size_t)slot * kM + mi) * p.head_size;
#pragma unroll
                for (int i = 0; i < HS / 8; ++i) {
                    const int d = 8 * i + 2 * t4;
                    if (d < p.head_size) *reinterpret_cast<float2 *>(dst + d) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
                }
            }
        }
        __syncwarp();  // the stage is read before the next copy into it
    }
    cp_wait<0>();
}

}  // namespace

// TC: blocks below the plan's share take the tensor-core role, the others walk.  Calls that have no use for it have a kernel of
// the walk alone, of fewer threads, which is up sooner.
template <typename T, int HS, bool BF, bool TC>
__global__ void __launch_bounds__(attn_threads(TC), 1) attn_pages_16_kernel(const __grid_constant__ TcAttn ta) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const PagesAttn &p = ta.p;
    pdl_launch_dependents();
    pdl_wait();
    const Plan pl = plan_here<attn_threads(TC)>(p, smem + kWork<HS, TC>, smem, blockIdx.x == 0);
    const int n_tc = TC ? pl.hdr[kHdrTcBlocks] : 0, warp = threadIdx.x / 32 - walk_first(TC);
    if constexpr (TC) {
        if ((int)blockIdx.x < n_tc) return tc_role<HS, BF>(ta, pl, smem, blockIdx.x);
        // the four warps that do not walk leave their registers to the eight that do: 24 + 2 * 240 = 3 * 168
        if (warp < 0) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 24;");
            return;
        }
        asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
    }
    walk_role<T, HS>(p, pl, smem, warp, n_tc);
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

template <typename T, int HS, bool BF, bool TC>
cudaError_t launch(const TcAttn &ta, cudaLaunchConfig_t cfg) {
    constexpr int bytes = kWork<HS, TC> + (int)kPlanSmem;
    auto fn = attn_pages_16_kernel<T, HS, BF, TC>;
    static DeviceOnce once;
    cudaError_t e = once.smem(reinterpret_cast<const void *>(fn), bytes, TC ? 168 : 0);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(ta.p.num_sms);
    cfg.blockDim = dim3(attn_threads(TC));
    cfg.dynamicSmemBytes = bytes;
    return cudaLaunchKernelEx(&cfg, fn, ta);
}
template <typename T, int HS, bool BF>
cudaError_t launch(const TcAttn &ta, cudaLaunchConfig_t cfg) {
    return ta.p.tc ? launch<T, HS, BF, true>(ta, cfg) : launch<T, HS, BF, false>(ta, cfg);
}

}  // namespace

// A box must start at a page row and cover whole groups of 8 lines of the swizzle: pages of 8 rows and more that divide a
// tile or are a multiple of one; a tensor's strides are below 2^40 bytes.
bool attn_pages_tc_supported(const PagesAttn &p) {
    const long long lim = 1ll << 40;
    return p.page_size >= 8 && (p.page_size % tc_keys(false) == 0 || tc_keys(false) % p.page_size == 0) && p.row_stride < lim && p.head_stride < lim &&
           p.page_stride < lim && tensor_map_encoder();
}

int attn_pages_16_shift(int hs) { return hs <= 64 ? 5 : 4; }
static_assert(Shape<64>::KT == 1 << 5 && Shape<128>::KT == 1 << 4, "the plan counts tiles by shifts");

cudaError_t launch_attn_pages_16(const PagesAttn &p, cudaLaunchConfig_t cfg) {
    TcAttn ta{};
    ta.p = p;
    ta.box_rows = p.page_size < tc_keys(false) ? p.page_size : tc_keys(false);
    ta.scale_log2 = p.scale_log2 < 0.f ? -p.scale_log2 : p.scale_log2;
    ta.flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    if (p.tc && (!encode_pages(&ta.kmap, p.k, p, ta.box_rows) || !encode_pages(&ta.vmap, p.v, p, ta.box_rows))) return cudaErrorInvalidValue;
    if (p.head_size <= 64) return p.dtype == L2_BF16 ? launch<TBf16, 64, true>(ta, cfg) : launch<TF16, 64, false>(ta, cfg);
    return p.dtype == L2_BF16 ? launch<TBf16, 128, true>(ta, cfg) : launch<TF16, 128, false>(ta, cfg);
}

}  // namespace l2
