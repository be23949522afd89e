// Rules on logits before sampling: penalties for tokens that a sequence holds already, biases, grammar masks.
//
// What it computes, for the logit l of token v in a row of sequence s (in fp32):
//     seen:     v is in the sequence's history, or on the row's own path of drafted tokens;
//     n:        how often, counting the history from counted_from[s] on;
//     l -> l / repetition[s] where l > 0, else l * repetition[s], if seen (the quotient as a product with the rounded inverse, two
//          roundings: within 2^-23 of the quotient; a division for each logit that is seen bounds the slices of frequent tokens);
//     l -> l - (frequency[s] n + presence[s]) if n > 0;
//     l -> l + the value of the sequence's last bias entry of v, if it has one;
//     l -> -inf where the row's mask has bit v clear.
//
// How.  Each logit is read and written once, which bounds it where there are many; a small call is a chain of dependent loads.
// A block takes a slice of the vocabulary and some rows.  It counts the sequence's history into a table of the slice in shared
// memory (integer atomics: the result does not depend on their order), once for all of its rows of that sequence: the history is
// read once for every slice, from L2.  An entry is the count (24 bits), whether the token is only seen (before counted_from), and, for a
// token that the tree drafted, the place of the first drafted token of that kind: its word in `kinds` says which of the
// tree's tokens are of the kind, so that a row adds those that are on its path (its word of the tree) to the count, and no row
// waits for another.  (480 rows of 30-token trees over 128000 tokens, bf16 to fp32: 79 us, 4.7 TB/s; with paths added to the table and
// taken off again, two barriers a row, 187.)  A bias table holds the number of the last entry of each token, by atomicMax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <type_traits>

#include "../../include/l2.h"
#include "l2_device.cuh"
#include "l2_pages.h"
#include "l2_rows.h"
#include "l2_tree.cuh"

namespace l2 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlice = 8192;   // tokens of a block: two tables of 32 KB
constexpr int kMinSlice = 1024;
constexpr int kMostRows = 32;     // rows of a block, where they come in trees
constexpr float kTableRows = 4.f; // what making the tables takes, in rows
// Blocks of an SM: as many as registers allow (80 a thread where an access has 8 elements, with 40 bytes of spills, 94 with biases), and with
// biases no more than two tables of the largest slice leave room for.
constexpr int reg_blocks(int width) { return width == 8 ? 3 : 4; }
constexpr int blocks_of(int width, bool bias) { return bias ? 3 : reg_blocks(width); }
constexpr unsigned kSeen = 1u << 31, kCount = (1u << 24) - 1;
constexpr int kKindShift = 24;    // 7 bits: 1 + the place
constexpr unsigned kKind = 0x7fu << kKindShift;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float x, float &y) { y = x; }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16 &y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(float x, __half &y) { y = __float2half_rn(x); }

template <typename T, int W>
struct alignas(sizeof(T) * W) Piece {
    T v[W];
};

}  // namespace

// TI, TO: types of logits and results; W: elements an access; BIAS: the call has biases (a second table).
template <typename TI, typename TO, int W, bool BIAS>
__global__ void __launch_bounds__(kThreads, reg_blocks(W)) rules_kernel(const RulesParams p) {
    extern __shared__ __align__(16) unsigned count[];  // [slice], and [slice] numbers of bias entries
    __shared__ u64 words[kTreeNodes], kinds[kTreeNodes];
    __shared__ int tokens[kTreeNodes], tree_ok;
    constexpr int K = W == 1 ? 8 : 4;  // accesses in flight a thread
    constexpr int kStep = K * W * kThreads;
    unsigned *entry = count + p.slice;
    const int tid = threadIdx.x, lane = tid & 31;
    const int v0 = blockIdx.y * p.slice, n_v = min(p.slice, p.vocab - v0);
    const int r0 = blockIdx.x * p.rows_per, r1 = min(r0 + p.rows_per, p.rows);
    pdl_launch_dependents();
    pdl_wait();
#pragma unroll 1
    for (int r = r0, end; r < r1; r = end) {
        // rows r .. end - 1 are of one tree: the last that starts at or before r
        int i = r, first = r;
        end = r + 1;
        bool good = true;
        if (p.starts) {
            int before = 0;
            for (int base = 0; base < p.n; base += kThreads) before += __syncthreads_count(base + tid < p.n && p.starts[base + tid] <= r);
            i = max(before - 1, 0);
            first = p.starts[i];
            const int b = p.starts[i + 1];
            if (r >= b && i == p.n - 1) return;  // rows behind the last tree are left as they are
            good = first >= 0 && first <= r && r < b && b <= p.rows && (!p.drafted || b - first <= kTreeNodes);
            if (good) end = b;
        }
        const int tree_end = end;
        end = min(end, r1);
        const int seq = p.seqs ? p.seqs[i] : i;
        good &= seq >= 0 && seq < p.n_seqs;
        int len = 0, counted = 0, b0 = 0, b1 = 0;
        float rep = 1.f, pres = 0.f, freq = 0.f;
        if (good) {
            len = p.lens[seq];
            if (p.counted) counted = p.counted[seq];
            if (p.repetition) rep = p.repetition[seq];
            if (p.presence) pres = p.presence[seq];
            if (p.frequency) freq = p.frequency[seq];
            if (BIAS) {
                b0 = p.bias_starts[seq];
                b1 = p.bias_starts[seq + 1];
            }
            good = len >= 0 && len <= p.max_len && b0 >= 0 && b0 <= b1 && b1 <= p.n_bias;
        }
        const float inv = 1.f / rep;
        const bool counting = good && !(rep == 1.f && pres == 0.f && freq == 0.f), biased = BIAS && good && b1 > b0;
        // a row's mask, nullptr for none; false if it is invalid
        auto mask_of = [&](int row, const unsigned *&mask) {
            const int m = p.masks ? (p.mask_rows ? p.mask_rows[row] : row) : -1;
            mask = m >= 0 ? p.masks + m * p.mask_stride + v0 / 32 : nullptr;
            return m >= -1 && m < max(p.n_masks, 0);
        };
        Piece<TI, W> x[K];
        unsigned bits[K];
        // whole: all of the block's accesses are, so that nothing is tested
        auto load = [&](auto whole, int row, const unsigned *mask, int base) {
            const TI *in = reinterpret_cast<const TI *>(p.logits + (long long)row * p.in_row) + v0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int v = base + (k * kThreads + tid) * W;
                bits[k] = ~0u;
                if (!decltype(whole)::value && v >= n_v) continue;
                if (decltype(whole)::value || W == 1 || v + W <= n_v)
                    x[k] = *reinterpret_cast<const Piece<TI, W> *>(in + v);
                else
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (v + e < n_v) x[k].v[e] = in[v + e];
                if (mask) bits[k] = mask[v >> 5] >> (v & 31);  // W divides 32: a piece's bits are of one word
            }
        };
        auto apply = [&](auto whole, int row, int base, u64 word) {
            TO *out = reinterpret_cast<TO *>(p.out + (long long)row * p.out_row) + v0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int v = base + (k * kThreads + tid) * W;
                if (!decltype(whole)::value && v >= n_v) continue;
                Piece<unsigned, W> c = {}, en = {};
                if (counting) c = *reinterpret_cast<const Piece<unsigned, W> *>(count + v);
                if (BIAS && biased) en = *reinterpret_cast<const Piece<unsigned, W> *>(entry + v);
                float l[W];
                unsigned some = 0;
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    l[e] = to_float(x[k].v[e]);
                    some |= c.v[e] | en.v[e];
                }
                if (some) {
                    // (without branches: where tokens are frequent, all of a warp's pieces come here)
                    if (some & kKind)
#pragma unroll
                        for (int e = 0; e < W; ++e)
                            if (c.v[e] & kKind) {
                                const unsigned mine = __popcll(kinds[(c.v[e] >> kKindShift & 0x7f) - 1] & word);
                                c.v[e] = (c.v[e] & ~kKind) + mine;  // the count has room: 2^24 - 1 - 64 tokens at most
                            }
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        const unsigned n = c.v[e] & kCount;
                        const float scale = l[e] > 0.f ? inv : rep, less = fmaf(freq, (float)n, pres);
                        l[e] = c.v[e] ? l[e] * scale : l[e];
                        l[e] = n ? l[e] - less : l[e];
                    }
                    if (BIAS && biased)
#pragma unroll
                        for (int e = 0; e < W; ++e)
                            if (en.v[e]) l[e] += p.bias_values[en.v[e] - 1];
                }
                Piece<TO, W> y;
#pragma unroll
                for (int e = 0; e < W; ++e) from_float(bits[k] >> e & 1u ? l[e] : -CUDART_INF_F, y.v[e]);
                if (decltype(whole)::value || W == 1 || v + W <= n_v)
                    *reinterpret_cast<Piece<TO, W> *>(out + v) = y;
                else
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (v + e < n_v) out[v + e] = y.v[e];
            }
        };
        // the first logits are on their way while the tables are made
        const unsigned *mask = nullptr;
        bool mask_good = mask_of(r, mask), loaded = good && mask_good;
        if (loaded) load(std::false_type(), r, mask, 0);
        __syncthreads();  // the tables before are read
        if (good && p.drafted && tid < kTreeNodes) {
            const int n = tree_end - first;
            tokens[tid] = tid < n ? p.drafted[first + tid] : -1;
            if (tid < 32) {
                const TreeParents t = tree_parents(p.starts && p.parents ? p.parents + first : nullptr, n);
                const TreeWords w = tree_words(t);
                words[lane] = w.lo;
                words[lane + 32] = w.hi;
                if (lane == 0) tree_ok = t.ok;
            }
        }
        if (counting)
            for (int v = tid * 4; v < p.slice; v += kThreads * 4) *reinterpret_cast<uint4 *>(count + v) = make_uint4(0u, 0u, 0u, 0u);
        if (biased)
            for (int v = tid * 4; v < p.slice; v += kThreads * 4) *reinterpret_cast<uint4 *>(entry + v) = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        if (good && p.drafted) good = tree_ok != 0;
        if (!good) {
            if (tid == 0 && p.err) atomicOr(p.err, L2_PAGES_ERR_ARGS);
            continue;
        }
        if (counting) {
            const int *h = p.history + seq * p.history_stride;
            constexpr int kAtOnce = 8;  // loads in flight
#pragma unroll 1
            for (int base = tid; base < len; base += kAtOnce * kThreads) {
                int t[kAtOnce];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) t[j] = base + j * kThreads < len ? h[base + j * kThreads] : -1;
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const unsigned u = (unsigned)t[j] - (unsigned)v0;
                    if (u >= (unsigned)n_v) continue;
                    if (base + j * kThreads >= counted)
                        atomicAdd(count + u, 1u);
                    else
                        atomicOr(count + u, kSeen);
                }
            }
            if (p.drafted && tid < kTreeNodes) {
                const unsigned u = (unsigned)tokens[tid] - (unsigned)v0;
                if (first + tid < tree_end && u < (unsigned)n_v) {
                    u64 same = 0;
                    for (int j = 0; j < tree_end - first; ++j) same |= (u64)(tokens[j] == tokens[tid]) << j;
                    kinds[tid] = same;
                    if (__ffsll(same) - 1 == tid) atomicOr(count + u, (unsigned)(tid + 1) << kKindShift);
                }
            }
        }
        if (biased)
            for (int e = b0 + tid; e < b1; e += kThreads) {
                const unsigned u = (unsigned)p.bias_tokens[e] - (unsigned)v0;
                if (u < (unsigned)n_v) atomicMax(entry + u, (unsigned)e + 1u);
            }
        __syncthreads();
#pragma unroll 1
        for (int row = r; row < end; ++row) {
            if (row > r) mask_good = mask_of(row, mask);
            if (!mask_good) {  // reported, and not written
                if (tid == 0 && p.err) atomicOr(p.err, L2_PAGES_ERR_ARGS);
                continue;
            }
            const u64 word = p.drafted ? words[row - first] : 0;
#pragma unroll 1
            for (int base = 0; base < n_v; base += kStep) {
                if (base + kStep <= n_v) {
                    if (!loaded) load(std::true_type(), row, mask, base);
                    apply(std::true_type(), row, base, word);
                } else {
                    if (!loaded) load(std::false_type(), row, mask, base);
                    apply(std::false_type(), row, base, word);
                }
                loaded = false;
            }
        }
    }
}

namespace {

template <typename TI, typename TO, int W, bool BIAS>
cudaError_t launch(const RulesParams &p, cudaLaunchConfig_t cfg) {
    auto fn = rules_kernel<TI, TO, W, BIAS>;
    cfg.dynamicSmemBytes = (BIAS ? 2 : 1) * p.slice * sizeof(unsigned);
    static DeviceOnce once;
    cudaError_t e = once.smem(reinterpret_cast<const void *>(fn), 2 * kMaxSlice * (int)sizeof(unsigned));
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, fn, p);
}
template <typename TI, typename TO>
cudaError_t launch(const RulesParams &p, int vec, cudaLaunchConfig_t cfg) {
    if constexpr (sizeof(TI) == 2 && sizeof(TO) == 2)
        if (vec == 8) return p.n_bias > 0 ? launch<TI, TO, 8, true>(p, cfg) : launch<TI, TO, 8, false>(p, cfg);
    if (vec >= 4) return p.n_bias > 0 ? launch<TI, TO, 4, true>(p, cfg) : launch<TI, TO, 4, false>(p, cfg);
    return p.n_bias > 0 ? launch<TI, TO, 1, true>(p, cfg) : launch<TI, TO, 1, false>(p, cfg);
}

}  // namespace

cudaError_t launch_rules(RulesParams p, int dtype, bool out_f32, int vec, int num_sms, cudaStream_t s) {
    if (p.rows == 0) return cudaSuccess;
    // The largest slice, since each counts the history anew, that still gives every SM blocks; rows of trees (on average rows / n) as many to
    // a block as make rounds of blocks over the SMs times a block's rows least, a table counting as kTableRows of them.  (480 rows of 128000, bf16: with
    // rounds of three blocks an SM, which is what there is room for, 76 us, with biases 104, to fp32 98; with rounds of four 89, 132, 116.)
    const int at_once = blocks_of(vec, p.n_bias > 0) * num_sms;
    p.rows_per = 1;
    p.slice = kMaxSlice;
    auto slices = [&]() { return (p.vocab + p.slice - 1) / p.slice; };
    if (p.rows >= 2 * p.n) {
        float least = 0.f;
        const float tree = (float)p.rows / (float)p.n;
        for (int r = 1; r <= kMostRows; ++r) {
            const long long blocks = (long long)slices() * ((p.rows + r - 1) / r), rounds = (blocks + at_once - 1) / at_once;
            const float cost = (float)rounds * ((float)r + kTableRows * (1.f + (float)(r - 1) / tree));
            if (r == 1 || cost < least) {
                least = cost;
                p.rows_per = r;
            }
        }
    }
    while ((long long)slices() * ((p.rows + p.rows_per - 1) / p.rows_per) * 2 <= 5ll * num_sms && p.slice > kMinSlice) p.slice /= 2;
    cudaLaunchConfig_t cfg = {};
    // slices one after the other: the first ones, whose tokens are as a rule the frequent ones, take longest
    cfg.gridDim = dim3((p.rows + p.rows_per - 1) / p.rows_per, (p.vocab + p.slice - 1) / p.slice);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (dtype == L2_F32) return launch<float, float>(p, vec, cfg);
    if (dtype == L2_BF16) return out_f32 ? launch<__nv_bfloat16, float>(p, vec, cfg) : launch<__nv_bfloat16, __nv_bfloat16>(p, vec, cfg);
    return out_f32 ? launch<__half, float>(p, vec, cfg) : launch<__half, __half>(p, vec, cfg);
}

}  // namespace l2
