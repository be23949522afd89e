// Acceptance of drafted tokens in a paged cache: of the rows that a sequence's tree of drafted tokens left behind its committed
// ones, those of one path from the root stay, side by side in every layer; the others' pages are given back.
//
// The path, where it is found here: token 0 (what was sampled after the committed rows); then, from each accepted token u on,
// the first child whose token is targets[u], what the model says follows u.  Parents come before their children, so a path is a
// set of ascending tokens: one 64-bit word.
//
// Two kernels, as for the other calls that move rows (pages.cu).  One block checks the whole call, finds the paths
// and changes counts and lengths only if everything fits: its cost is the latency of a chain of dependent loads, the walk down a
// tree is in registers (a child is found by a ballot).  Then a grid moves the rows, bound by HBM: a thread takes one 16-byte word of
// a (layer, K or V, head) through the path in batches of eight, loads before stores.  The j-th row of a path goes to place j and comes from place
// path[j] >= j, so what a batch writes is no later batch's source.  (16 trees of 40 to 64 tokens, up to nine accepted, 32 layers of the 7B shape in bf16:
// 15 us, about half of it the books.)
#include <cuda_runtime.h>

#include "l2_device.cuh"
#include "l2_pages.h"
#include "l2_tree.cuh"

namespace l2 {

namespace {

constexpr int kT = kPagesThreads;
constexpr int kMoveThreads = 256;
constexpr int kBatch = 8;
// Up to so many words of a position, of all sequences, the first kernel moves them itself: a launch less.
constexpr int kMoveHere = 4096;

__device__ __forceinline__ int ceil_div_d(int a, int b) { return (a + b - 1) / b; }
__device__ __forceinline__ bool page_ok(const PagesView &p, int page) { return page >= 0 && page < p.n_pages; }
// Ends a refused call: nothing was changed, the kernel that moves rows skips, and what is found says that nothing is accepted.
__device__ __forceinline__ void refuse(const PagesView &p, const PagesAccept &a, int bit) {
    const int i = threadIdx.x;
    if (i == 0) {
        atomicOr(p.err, bit);
        p.scratch[kScrRefused] = 1;
    }
    if (!a.find) return;
    for (int r = i; r < a.rows; r += kT) a.path[r] = -1;
    if (i < a.n) {
        a.counts[i] = 0;
        if (a.next) a.next[i] = -1;
    }
}

// The accepted tokens of a tree of n (1..64) tokens, by a warp; *last: the last of them.
__device__ __forceinline__ u64 walk_path(const TreeParents &t, const int *tokens, const int *targets, int n, int *last) {
    const int lane = threadIdx.x & 31;
    const int tok_lo = lane < n ? tokens[lane] : 0, tok_hi = lane + 32 < n ? tokens[lane + 32] : 0;
    const int tar_lo = lane < n ? targets[lane] : 0, tar_hi = lane + 32 < n ? targets[lane + 32] : 0;
    u64 path = 1;
    int u = 0;
#pragma unroll 1
    while (true) {  // u rises, so at most n rounds
        const int a = __shfl_sync(0xffffffffu, tar_lo, u & 31), b = __shfl_sync(0xffffffffu, tar_hi, u & 31), want = u < 32 ? a : b;
        const unsigned lo = __ballot_sync(0xffffffffu, lane < n && t.lo == u && tok_lo == want);
        const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 < n && t.hi == u && tok_hi == want);
        if (!(lo | hi)) break;
        u = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
        path |= 1ull << u;
    }
    *last = u;
    return path;
}

// Byte offset, in a (layer, K or V, head), of a sequence's row.
__device__ __forceinline__ long long row_offset(const PagesView &p, int s, int pos) {
    const int col = (int)((unsigned)pos / (unsigned)p.page_size);
    return p.table[(size_t)s * p.max_pages + col] * p.page_stride + (pos - col * p.page_size) * p.row_stride;
}

// Moves word u of all (layer, K or V, head) words along a path of c tokens whose first `stay` are where they were.
template <class From, class To>
__device__ __forceinline__ void move_word(const PagesView &p, long long u, int stay, int c, From from, To to) {
    const int vh = p.row_bytes >> 4, words = vh * p.n_kv_heads;
    const int w = (int)(u % words), lv = (int)(u / words), h = w / vh;
    char *pool = (lv & 1 ? p.v : p.k) + (lv >> 1) * p.layer_stride + h * p.head_stride + ((w - h * vh) << 4);
#pragma unroll 1
    for (int j0 = stay; j0 < c; j0 += kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (j0 + j < c) x[j] = *reinterpret_cast<const uint4 *>(pool + from(j0 + j));
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (j0 + j < c) *reinterpret_cast<uint4 *>(pool + to(j0 + j)) = x[j];
    }
}

}  // namespace

__global__ void __launch_bounds__(kT) pages_accept_kernel(const PagesView p, const PagesAccept a) {
    __shared__ int sq[kPagesMaxCall], first_s[kPagesMaxCall], n_s[kPagesMaxCall], len_s[kPagesMaxCall], last_s[kPagesMaxCall], why;
    __shared__ u64 path_s[kPagesMaxCall];
    __shared__ long long from[kTreeNodes], to[kTreeNodes];  // byte offsets of rows, where this block moves them
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int s = i < a.n ? a.seqs[i] : -1;
    sq[i] = s;
    if (i == 0) why = 0;
    __syncthreads();
    bool bad = false;
    int end = -1;  // page that the sequence ends in
    if (i < a.n) {
        const int b0 = a.starts[i], b1 = a.starts[i + 1];
        bad = s < 0 || s >= p.n_seqs || b0 < 0 || b1 < b0 || b1 > a.rows || b1 - b0 > kTreeNodes || (i == 0 && b0 != 0);
        for (int j = 0; j < i; ++j) bad |= sq[j] == s;
        int len = 0;
        if (!bad) {
            len = p.lens[s];
            bad = len < b1 - b0 || len > (long long)p.max_pages * p.page_size;
            if (!bad && b1 > b0) end = p.table[(size_t)s * p.max_pages + (len - 1) / p.page_size];
        }
        first_s[i] = b0;
        n_s[i] = b1 - b0;
        len_s[i] = len;
    }
    if (__syncthreads_or(bad)) return refuse(p, a, L2_PAGES_ERR_ARGS);
    // whether its last rows are others than the tree's (see PagesView::missing), which is known when the paths are
    const bool without_rows = page_ok(p, end) && p.missing()[end];
    // the paths, a warp each
    for (int e = warp; e < a.n; e += kT / 32) {
        const int n = n_s[e], first = first_s[e];
        u64 path = 0;
        int last = -1;
        if (a.find) {
            const TreeParents t = tree_parents(a.parents ? a.parents + first : nullptr, n);
            bad |= !t.ok;
            if (n && t.ok) path = walk_path(t, a.tokens + first, a.targets + first, n, &last);
        } else {
            const int c = a.counts[e];
            bad |= c < 0 || c > n;
            if (c >= 0 && c <= n) {
                unsigned lo = 0, hi = 0;
                int before = -1;
                for (int j0 = 0; j0 < c; j0 += 32) {
                    const int j = j0 + lane, x = j < c ? a.path[first + j] : kTreeNodes;
                    int prev = __shfl_up_sync(0xffffffffu, x, 1);
                    if (lane == 0) prev = before;
                    const bool fine = j >= c || (x > prev && x < n);
                    bad |= !__all_sync(0xffffffffu, fine);
                    lo |= __reduce_or_sync(0xffffffffu, j < c && fine && x < 32 ? 1u << x : 0u);
                    hi |= __reduce_or_sync(0xffffffffu, j < c && fine && x >= 32 ? 1u << (x - 32) : 0u);
                    before = __shfl_sync(0xffffffffu, x, 31);
                }
                path = (u64)hi << 32 | lo;
            }
        }
        if (lane == 0) {
            path_s[e] = path;
            last_s[e] = last;
        }
    }
    if (__syncthreads_or(bad || without_rows)) return refuse(p, a, L2_PAGES_ERR_ARGS);
    // pages that rows move into, and the partly filled last one, must be the sequence's alone; those that rows come from and those
    // that are given back must exist
    for (int e = warp; e < a.n; e += kT / 32) {
        const u64 path = path_s[e];
        const int n = n_s[e], c = __popcll(path), base = len_s[e] - n, now = base + c;
        if (c == n) continue;  // nothing moves or goes
        const int *t = p.table + (size_t)sq[e] * p.max_pages;
        const int stay = min(c, __ffsll(~path) - 1);  // tokens 0 .. stay - 1 are where they were (~path is not 0: c < n)
        const int c0 = base / p.page_size, c1 = ceil_div_d(len_s[e], p.page_size);
        for (int col = c0 + lane; col < c1; col += 32) {
            const int page = t[col];
            if (!page_ok(p, page)) {
                atomicOr(&why, L2_DEV_ERR_BOUNDS);
                continue;
            }
            const int lo = col * p.page_size, hi = lo + p.page_size;  // its positions
            const bool moved_into = base + stay < now && base + stay < hi && lo < now;
            const bool part = lo < now && now < hi;
            if ((moved_into || part) && p.refs[page] != 1) atomicOr(&why, L2_PAGES_ERR_ARGS);
        }
    }
    __syncthreads();
    if (const int w = why) return refuse(p, a, w);
    __syncthreads();  // every warp has read it before it may be set again
    auto gone = [&](auto take) {  // every page that is given back
        for (int e = warp; e < a.n; e += kT / 32) {
            const int now = len_s[e] - n_s[e] + __popcll(path_s[e]), c1 = ceil_div_d(len_s[e], p.page_size);
            const int *t = p.table + (size_t)sq[e] * p.max_pages;
            for (int col = ceil_div_d(now, p.page_size) + lane; col < c1; col += 32) take(t[col]);
        }
    };
    gone([&](int page) {
        if (atomicSub(p.refs + page, 1) <= 0) atomicOr(&why, L2_PAGES_ERR_ARGS);  // no holder left
    });
    __syncthreads();
    if (why) {  // nothing changes: what was taken is put back
        gone([&](int page) { atomicAdd(p.refs + page, 1); });
        return refuse(p, a, why);
    }
    for (int e = warp; e < a.n; e += kT / 32) {
        const u64 path = path_s[e];
        const int n = n_s[e], first = first_s[e], c = __popcll(path);
        if (lane == 0) p.lens[sq[e]] = len_s[e] - n + c;
        if (!a.find) continue;
        for (int j = lane; j < n; j += 32) {  // token j is the popc-th of the path, or entry c + .. is free
            const int before = __popcll(path & ((1ull << j) - 1));
            if (path >> j & 1)
                a.path[first + before] = j;
            else
                a.path[first + c + j - before] = -1;
        }
        if (lane == 0) {
            a.counts[e] = c;
            if (a.next) a.next[e] = n ? a.targets[first + last_s[e]] : -1;
        }
    }
    if (a.find)  // rows behind the last tree
        for (int r = first_s[a.n - 1] + n_s[a.n - 1] + i; r < a.rows; r += kT) a.path[r] = -1;
    if (i == 0) p.scratch[kScrRefused] = 0;
    if (!a.move_here) return;
    // little to move: this block does it
    const int words = 2 * p.n_layers * p.n_kv_heads * (p.row_bytes >> 4);
    for (int e = 0; e < a.n; ++e) {
        const u64 path = path_s[e];
        const int n = n_s[e], c = __popcll(path), s0 = sq[e], base = len_s[e] - n, stay = min(c, __ffsll(~path) - 1);
        if (c == n || stay == c) continue;
        __syncthreads();  // the offsets before are read
        if (i < n && (path >> i & 1)) from[__popcll(path & ((1ull << i) - 1))] = row_offset(p, s0, base + i);
        if (i < c) to[i] = row_offset(p, s0, base + i);
        __syncthreads();
        for (int u = i; u < words; u += kT) move_word(p, u, stay, c, [&](int j) { return from[j]; }, [&](int j) { return to[j]; });
    }
}

// Block (x, i) moves its share of the words of sequence seqs[i]'s rows.
__global__ void __launch_bounds__(kMoveThreads) pages_accept_move_kernel(const PagesView p, const PagesAccept a) {
    __shared__ long long from[kTreeNodes], to[kTreeNodes];  // byte offsets of rows
    __shared__ int stay_s;
    pdl_launch_dependents();
    pdl_wait();
    if (p.scratch[kScrRefused]) return;
    const int i = blockIdx.y, tid = threadIdx.x;
    const int s = a.seqs[i], first = a.starts[i], c = a.counts[i], n = a.starts[i + 1] - first;
    if (c == 0 || c == n) return;
    const int base = p.lens[s] - c;
    if (tid == 0) stay_s = c;
    __syncthreads();
    if (tid < c) {
        const int x = a.path[first + tid];
        from[tid] = row_offset(p, s, base + x);
        to[tid] = row_offset(p, s, base + tid);
        if (x != tid) atomicMin(&stay_s, tid);  // from here on rows move: the path is ascending
    }
    __syncthreads();
    const long long u = (long long)blockIdx.x * kMoveThreads + tid;
    if (u < 2ll * p.n_layers * p.n_kv_heads * (p.row_bytes >> 4)) move_word(p, u, stay_s, c, [&](int j) { return from[j]; }, [&](int j) { return to[j]; });
}

cudaError_t launch_pages_accept(const PagesView &p, PagesAccept a, cudaStream_t s) {
    const long long words = 2ll * p.n_layers * p.n_kv_heads * (p.row_bytes >> 4);
    a.move_here = words * a.n <= kMoveHere;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kT);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pages_accept_kernel, p, a);
    if (e != cudaSuccess || a.rows == 0 || a.move_here) return e;
    cfg.gridDim = dim3((unsigned)((words + kMoveThreads - 1) / kMoveThreads), a.n);
    cfg.blockDim = dim3(kMoveThreads);
    return cudaLaunchKernelEx(&cfg, pages_accept_move_kernel, p, a);
}

}  // namespace l2
