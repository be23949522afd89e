// Rules on logits before sampling: penalties for tokens that a sequence holds already, biases, grammar masks.
//
// What it computes, for the logit l of token v in a row of sequence s (in fp32):
//     seen:     v is in the sequence's history, or on the row's own path of drafted tokens;
//     n:        how often, counting the history from counted_from[s] on;
//     l -> l / repetition[s] where l > 0, else l * repetition[s], if seen;
//     l -> l - (frequency[s] n + presence[s]) if n > 0;
//     l -> l + the value of the sequence's last bias entry of v, if it has one;
//     l -> -inf where the row's mask has bit v clear.
//
// How.  Each logit is read and written once, which bounds it where there are many; a small call is a chain of dependent loads.
// A block takes a slice of the vocabulary and some rows.  It counts the sequence's history into a table of the slice in shared
// memory (integer atomics: the result does not depend on their order), once for all of its rows of that sequence: the history is
// read once for every slice, from L2.  A row's own path, at most 64 tokens, is added before the row and taken off again after it.
// Bit 31 of a count says that the token is only seen (before counted_from); a bias table holds the number of the last
// entry of each token, by atomicMax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

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
constexpr int kRowsPer = 8;       // most rows of a block
constexpr unsigned kSeen = 1u << 31;

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
__global__ void __launch_bounds__(kThreads) rules_kernel(const RulesParams p) {
    extern __shared__ __align__(16) unsigned count[];  // [slice], and [slice] numbers of bias entries
    __shared__ u64 words[kTreeNodes];
    __shared__ int tree_ok;
    unsigned *entry = count + p.slice;
    const int tid = threadIdx.x, lane = tid & 31;
    const int v0 = blockIdx.x * p.slice, n_v = min(p.slice, p.vocab - v0);
    const int r0 = blockIdx.y * p.rows_per, r1 = min(r0 + p.rows_per, p.rows);
    pdl_launch_dependents();
    pdl_wait();
    int at = -1, first = 0, end = 0, seq = 0;  // the tree whose tables are up: its number, rows, sequence
    bool good = false, counting = false, biased = false;
    float rep = 1.f, pres = 0.f, freq = 0.f;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        if (at < 0 || r >= end) {
            // the row's tree: the last that starts at or before it
            int i = r, a = r, b = r + 1;
            if (p.starts) {
                int lo = 0, hi = p.n;
                while (hi - lo > 1) {
                    const int m = (lo + hi) >> 1;
                    p.starts[m] <= r ? lo = m : hi = m;
                }
                i = lo;
                a = p.starts[i];
                b = p.starts[i + 1];
                if (r >= b && i == p.n - 1) return;  // rows behind the last tree are left as they are
            }
            at = i;
            first = a;
            seq = p.seqs ? p.seqs[i] : i;
            good = a >= 0 && a <= r && r < b && b <= p.rows && seq >= 0 && seq < p.n_seqs && (!p.drafted || b - a <= kTreeNodes);
            end = a <= r && r < b ? b : r + 1;
            int len = 0, counted = 0, b0 = 0, b1 = 0;
            if (good) {
                len = p.lens[seq];
                counted = p.counted ? p.counted[seq] : 0;
                rep = p.repetition ? p.repetition[seq] : 1.f;
                pres = p.presence ? p.presence[seq] : 0.f;
                freq = p.frequency ? p.frequency[seq] : 0.f;
                good = len >= 0 && len <= p.max_len;
                if (BIAS) {
                    b0 = p.bias_starts[seq];
                    b1 = p.bias_starts[seq + 1];
                    good &= b0 >= 0 && b0 <= b1 && b1 <= p.n_bias;
                }
            }
            counting = good && !(rep == 1.f && pres == 0.f && freq == 0.f);
            biased = BIAS && good && b1 > b0;
            __syncthreads();  // the tables before are read
            if (good && p.drafted && tid < 32) {
                const TreeParents t = tree_parents(p.parents ? p.parents + first : nullptr, end - first);
                const TreeWords w = tree_words(t);
                words[lane] = w.lo;
                words[lane + 32] = w.hi;
                if (lane == 0) tree_ok = t.ok;
            }
            if (counting)
                for (int v = tid * 4; v < p.slice; v += kThreads * 4) *reinterpret_cast<uint4 *>(count + v) = make_uint4(0u, 0u, 0u, 0u);
            if (biased)
                for (int v = tid * 4; v < p.slice; v += kThreads * 4) *reinterpret_cast<uint4 *>(entry + v) = make_uint4(0u, 0u, 0u, 0u);
            __syncthreads();
            if (good && p.drafted) good = tree_ok != 0;
            if (counting) {
                const int *h = p.history + seq * p.history_stride;
#pragma unroll 4
                for (int j = tid; j < len; j += kThreads) {
                    const unsigned u = (unsigned)h[j] - (unsigned)v0;
                    if (u < (unsigned)n_v) {
                        if (j >= counted)
                            atomicAdd(count + u, 1u);
                        else
                            atomicOr(count + u, kSeen);
                    }
                }
            }
            if (biased)
                for (int e = b0 + tid; e < b1; e += kThreads) {
                    const unsigned u = (unsigned)p.bias_tokens[e] - (unsigned)v0;
                    if (u < (unsigned)n_v) atomicMax(entry + u, (unsigned)e + 1u);
                }
            __syncthreads();
        }
        const int mask_row = p.masks ? (p.mask_rows ? p.mask_rows[r] : r) : -1;
        if (!good || mask_row < -1 || mask_row >= max(p.n_masks, 0)) {  // reported, and not written
            if (tid == 0 && p.err) atomicOr(p.err, L2_PAGES_ERR_ARGS);
            continue;
        }
        // the row's own path
        const bool path = counting && p.drafted;
        const int mine = r - first;
        auto on_path = [&](unsigned d) {
            if (tid < kTreeNodes && first + tid < end && (words[mine] >> tid & 1)) {
                const unsigned u = (unsigned)p.drafted[first + tid] - (unsigned)v0;
                if (u < (unsigned)n_v) atomicAdd(count + u, d);
            }
        };
        if (path) {
            on_path(1u);
            __syncthreads();
        }
        const TI *in = reinterpret_cast<const TI *>(p.logits + (long long)r * p.in_row) + v0;
        TO *out = reinterpret_cast<TO *>(p.out + (long long)r * p.out_row) + v0;
        const unsigned *mask = mask_row < 0 ? nullptr : p.masks + mask_row * p.mask_stride + v0 / 32;
        auto rule = [&](float l, unsigned c, unsigned e, bool allowed) {
            if (counting && c) {
                l = l > 0.f ? l / rep : l * rep;
                const unsigned n = c & ~kSeen;
                if (n) l -= fmaf(freq, (float)n, pres);
            }
            if (biased && e) l += p.bias_values[e - 1];
            return allowed ? l : -CUDART_INF_F;
        };
        constexpr int K = W == 1 ? 8 : 4;  // accesses in flight a thread
#pragma unroll 1
        for (int base = 0; base < n_v; base += K * W * kThreads) {
            Piece<TI, W> x[K];
            unsigned bits[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int v = base + (k * kThreads + tid) * W;
                bits[k] = ~0u;
                if (v >= n_v) continue;
                if (W == 1 || v + W <= n_v)
                    x[k] = *reinterpret_cast<const Piece<TI, W> *>(in + v);
                else
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (v + e < n_v) x[k].v[e] = in[v + e];
                if (mask) bits[k] = mask[v >> 5] >> (v & 31);  // W divides 32: a piece's bits are of one word
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int v = base + (k * kThreads + tid) * W;
                if (v >= n_v) continue;
                Piece<unsigned, W> c = {}, en = {};
                if (counting) c = *reinterpret_cast<const Piece<unsigned, W> *>(count + v);
                if (BIAS && biased) en = *reinterpret_cast<const Piece<unsigned, W> *>(entry + v);
                Piece<TO, W> y;
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (W == 1 || v + e < n_v) from_float(rule(to_float(x[k].v[e]), c.v[e], en.v[e], bits[k] >> e & 1u), y.v[e]);
                if (W == 1 || v + W <= n_v)
                    *reinterpret_cast<Piece<TO, W> *>(out + v) = y;
                else
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (v + e < n_v) out[v + e] = y.v[e];
            }
        }
        if (path) {
            __syncthreads();
            on_path(~0u);  // - 1
            __syncthreads();
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
cudaError_t launch(const RulesParams &p, bool vec, cudaLaunchConfig_t cfg) {
    const bool bias = p.n_bias > 0;
    if (vec) return bias ? launch<TI, TO, 4, true>(p, cfg) : launch<TI, TO, 4, false>(p, cfg);
    return bias ? launch<TI, TO, 1, true>(p, cfg) : launch<TI, TO, 1, false>(p, cfg);
}

}  // namespace

cudaError_t launch_rules(RulesParams p, int dtype, bool out_f32, bool vec, int num_sms, cudaStream_t s) {
    if (p.rows == 0) return cudaSuccess;
    // the largest slice, and trees' rows together, as long as there are blocks for every SM several times over
    p.rows_per = p.starts ? kRowsPer : 1;
    p.slice = kMaxSlice;
    auto blocks = [&]() { return (long long)((p.vocab + p.slice - 1) / p.slice) * ((p.rows + p.rows_per - 1) / p.rows_per); };
    while (blocks() < 4ll * num_sms && p.rows_per > 1) p.rows_per /= 2;
    while (blocks() < 4ll * num_sms && p.slice > kMinSlice) p.slice /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.vocab + p.slice - 1) / p.slice, (p.rows + p.rows_per - 1) / p.rows_per);
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
