// Bookkeeping and row movement of a paged KV cache: append, read, fork, free, compact.
//
// A pool holds pages of page_size rows; a page belongs to refs[page] sequences, and
// sequence s of lens[s] rows holds pages table[s][0 .. ceil(lens[s] / page_size)).
// Pages are shared whole: a partly filled last page belongs to one sequence alone, so
// appending never writes a row that another sequence reads.
//
// Each call is one block that checks the whole call, finds the lowest free pages and
// changes counts, lengths and tables only when everything fits (otherwise it changes
// nothing and sets the pool's status word), and, where rows move, a grid that moves
// them.  The bookkeeping is a few thousand integers and its cost is the latency of a
// chain of dependent loads, so one block of 1024 threads is enough; free pages go out
// in ascending order and in the order of the call, so the result does not depend on
// timing.  The row kernels are bound by HBM: 16-byte words, each read and written once.
#include <cuda_runtime.h>

#include "l2_device.cuh"
#include "l2_pages.h"

namespace l2 {

namespace {

constexpr int kT = kPagesThreads;

__device__ __forceinline__ int ceil_div_d(int a, int b) { return (a + b - 1) / b; }

// Exclusive prefix sum over the block's threads; *total receives the sum.
__device__ __forceinline__ int block_scan(int v, int *total, int *buf) {
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
    *total = buf[32 + kT / 32 - 1];
    __syncthreads();
    return before + x - v;
}

// The `need` lowest free pages in ascending order into list; returns how many there are (at
// most need).  Four counts a thread and step, so a step takes 4096 pages.
__device__ int lowest_free(const PagesView &p, int need, int *list, int *buf) {
    int found = 0;
    for (int base = 0; base < p.n_pages && found < need; base += 4 * kT) {
        const int i0 = base + 4 * threadIdx.x;
        bool f[4];
        int c = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = i0 + j < p.n_pages && p.refs[i0 + j] == 0;
            c += f[j];
        }
        int total;
        int at = found + block_scan(c, &total, buf);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (f[j]) {
                if (at < need) list[at] = i0 + j;
                ++at;
            }
        found += total;
    }
    __syncthreads();  // the list is visible to the block
    return found < need ? found : need;
}

// Copies `words` 16-byte words, vr to a row and rows row_stride bytes apart, with NT threads, of which this is number t: W
// words in flight a thread (all loads before the stores, which might alias as far as the compiler knows).
template <int NT, int W>
__device__ __forceinline__ void copy_words(const char *a, char *b, int t, int words, int vr, long long row_stride) {
    const bool flat = row_stride == (long long)vr * 16;
#pragma unroll 1
    for (int c0 = t; c0 < words; c0 += W * NT) {
        uint4 x[W];
        long long o[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int c = c0 + j * NT;
            if (flat)
                o[j] = (long long)c << 4;
            else {
                const int r = (int)((unsigned)c / (unsigned)vr);
                o[j] = r * row_stride + ((long long)(c - r * vr) << 4);
            }
            if (c < words) x[j] = *reinterpret_cast<const uint4 *>(a + o[j]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (c0 + j * NT < words) *reinterpret_cast<uint4 *>(b + o[j]) = x[j];
    }
}

// Ends a refused call: nothing was changed, the row kernels that go by `flag` skip.
__device__ __forceinline__ void refuse(const PagesView &p, int bit, int flag = kScrRefused) {
    if (threadIdx.x == 0) {
        atomicOr(p.err, bit);
        p.scratch[flag] = 1;
    }
}

__device__ __forceinline__ bool page_ok(const PagesView &p, int page) { return page >= 0 && page < p.n_pages; }
__device__ __forceinline__ bool page_held(const PagesView &p, int page) { return page_ok(p, page) && p.refs[page] > 0; }

}  // namespace

// Append, first half: lens[seqs[i]] grows by its rows and takes the pages that needs, the
// lowest free ones in the order of i.
__global__ void __launch_bounds__(kT) pages_extend_kernel(const PagesView p, int n, const int *seqs, const int *starts, int rows) {
    __shared__ int buf[64], sq[kPagesMaxCall], base_s[kPagesMaxCall + 1];
    const int i = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const int s = i < n ? seqs[i] : -1;
    sq[i] = s;
    __syncthreads();
    bool bad = false;
    int old = 0, cnt = 0, have = 0, want = 0;
    if (i < n) {
        const int a = starts ? starts[i] : i, b = starts ? starts[i + 1] : i + 1;
        bad = s < 0 || s >= p.n_seqs || a < 0 || b < a || b > rows || (i == 0 && a != 0) || (i == n - 1 && b != rows);
        for (int j = 0; j < i; ++j) bad |= sq[j] == s;
        if (!bad) {
            old = p.lens[s];
            cnt = b - a;
            bad = old < 0 || (long long)old + cnt > (long long)p.max_pages * p.page_size;
        }
        if (!bad) {
            have = ceil_div_d(old, p.page_size);
            want = ceil_div_d(old + cnt, p.page_size);
            // rows go into a partly filled last page only if no other sequence holds it
            if (cnt > 0 && old % p.page_size) {
                const int page = p.table[(size_t)s * p.max_pages + have - 1];
                bad = !page_ok(p, page) || p.refs[page] != 1;
            }
        }
    }
    if (__syncthreads_or(bad)) return refuse(p, L2_PAGES_ERR_ARGS, kScrExtension);
    int need;
    const int base = block_scan(want - have, &need, buf);
    base_s[i] = base;
    if (i == 0) base_s[kT] = need;
    int *list = p.scratch + kScrHead;
    if (need > p.n_pages || lowest_free(p, need, list, buf) < need) return refuse(p, L2_PAGES_ERR_FULL, kScrExtension);
    // page e of the list belongs to the last sequence whose base is at most e and that takes pages
    for (int e = i; e < need; e += kT) {
        int lo = 0, hi = n;  // base_s[lo] <= e < base_s[hi]
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            (m < n ? base_s[m] : need) <= e ? lo = m : hi = m;
        }
        const int t = sq[lo], h = ceil_div_d(p.lens[t], p.page_size);
        const int page = list[e];
        p.table[(size_t)t * p.max_pages + h + e - base_s[lo]] = page;
        p.refs[page] = 1;
    }
    __syncthreads();  // the lengths above are read
    if (i < n) p.lens[s] = old + cnt;
    if (i == 0) p.scratch[kScrExtension] = 0;
}

// Append, second half: one warp per new row and layer range copies its heads' K and V.  A row's place
// is found once (its sequence, length, page: dependent loads) and used for every layer of the warp.
// READ: the other way, from the sequences' first rows.
template <bool READ>
__global__ void __launch_bounds__(256) pages_rows_kernel(const PagesView p, const PagesAppend a, int layers_per) {
    const int lane = threadIdx.x & 31;
    const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    const int groups = ceil_div_d(a.n_layers, layers_per);
    if (warp >= a.rows * groups) return;
    const int r = warp / groups, lg = warp - r * groups;
    if (!READ && p.scratch[kScrExtension]) return;
    int i = r, start = r, end = r + 1;
    if (a.starts) {
        int lo = 0, hi = a.n;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            a.starts[m] <= r ? lo = m : hi = m;
        }
        i = lo;
        start = a.starts[i];
        end = a.starts[i + 1];
    }
    const int s = a.seqs[i];
    const int n = s >= 0 && s < p.n_seqs ? p.lens[s] : -1;
    const int pos = n < 0 ? -1 : READ ? r - start : n - (end - r);
    if (READ && (r < start || r >= end || pos >= n)) {  // no such row
        if (lane == 0) atomicOr(p.err, L2_PAGES_ERR_ARGS);
        return;
    }
    int page = -1;
    if (r >= start && r < end && pos >= 0 && pos / p.page_size < p.max_pages)
        page = p.table[(size_t)s * p.max_pages + pos / p.page_size];
    if (!page_ok(p, page)) {
        if (lane == 0) atomicOr(p.err, L2_DEV_ERR_BOUNDS);
        return;
    }
    if (!READ && !a.extended && p.refs[page] != 1) {  // other sequences would see the row
        if (lane == 0) atomicOr(p.err, L2_PAGES_ERR_ARGS);
        return;
    }
    const long long at = page * p.page_stride + (pos % p.page_size) * p.row_stride;
    const int vh = p.row_bytes >> 4, nv = vh * p.n_kv_heads;  // 16-byte words a head, a row
    const int l0 = lg * layers_per, l1 = min(a.n_layers, l0 + layers_per);
    // four layers of K and V in flight a lane: their loads before the stores
    for (int c = lane; c < nv; c += 32) {
        const int h = c / vh, w = (c - h * vh) << 4;
        const long long so = (long long)r * a.row_stride + h * a.head_stride + w;
        const long long d = at + h * p.head_stride + w;
        for (int l = l0; l < l1; l += 4) {
            uint4 kx[4], vx[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (l + j < l1) {
                    const long long rows = so + (l + j) * a.layer_stride, pool = d + (a.layer0 + l + j) * p.layer_stride;
                    kx[j] = __ldcs(reinterpret_cast<const uint4 *>(READ ? p.k + pool : a.k + rows));
                    vx[j] = __ldcs(reinterpret_cast<const uint4 *>(READ ? p.v + pool : a.v + rows));
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (l + j < l1) {
                    const long long rows = so + (l + j) * a.layer_stride, pool = d + (a.layer0 + l + j) * p.layer_stride;
                    *reinterpret_cast<uint4 *>(READ ? a.k + rows : p.k + pool) = kx[j];
                    *reinterpret_cast<uint4 *>(READ ? a.v + rows : p.v + pool) = vx[j];
                }
        }
    }
}

// Fork, first half: sequence dst[i] becomes the first rows[i] rows of src[i] (all, without rows): whole
// pages by reference, a new page for what is left.
__global__ void __launch_bounds__(kT) pages_fork_kernel(const PagesView p, int n, const int *src, const int *dst, const int *rows) {
    __shared__ int buf[64], ss[kPagesMaxCall], sd[kPagesMaxCall], full_s[kPagesMaxCall];
    const int i = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const int s = i < n ? src[i] : -1, d = i < n ? dst[i] : -2;
    ss[i] = s;
    sd[i] = d;
    __syncthreads();
    bool bad = false;
    int m = 0;
    if (i < n) {
        bad = s < 0 || s >= p.n_seqs || d < 0 || d >= p.n_seqs;
        for (int j = 0; j < n; ++j) bad |= ss[j] == d || (j != i && sd[j] == d);
        if (!bad) {
            m = p.lens[s];
            bad = p.lens[d] != 0 || m < 0 || m > (long long)p.max_pages * p.page_size;
            if (rows && !bad) {
                bad = rows[i] < 0 || rows[i] > m;
                m = rows[i];
            }
        }
    }
    if (__syncthreads_or(bad)) return refuse(p, L2_PAGES_ERR_ARGS);
    const int full = m / p.page_size, tail = m % p.page_size;
    full_s[i] = full;
    // every page that would be shared or copied must exist and be held (one that is not might be handed out below)
    const int warp = i >> 5, lane = i & 31;
    __syncthreads();
    for (int e = warp; e < n; e += kT / 32) {
        const int *ts = p.table + (size_t)ss[e] * p.max_pages;
        for (int j = lane; j < full_s[e]; j += 32) bad |= !page_held(p, ts[j]);
    }
    if (i < n && tail) bad |= !page_held(p, p.table[(size_t)s * p.max_pages + full]);
    if (__syncthreads_or(bad)) return refuse(p, L2_PAGES_ERR_ARGS);
    int need;
    const int base = block_scan(i < n && tail ? 1 : 0, &need, buf);
    int *list = p.scratch + kScrHead;
    if (need > p.n_pages || lowest_free(p, need, list, buf) < need) return refuse(p, L2_PAGES_ERR_FULL);
    for (int e = warp; e < n; e += kT / 32) {
        const int *ts = p.table + (size_t)ss[e] * p.max_pages;
        int *td = p.table + (size_t)sd[e] * p.max_pages;
        for (int j = lane; j < full_s[e]; j += 32) {
            const int page = ts[j];
            td[j] = page;
            atomicAdd(p.refs + page, 1);
        }
    }
    if (i < n) {
        if (tail) {
            const int page = list[base];
            p.table[(size_t)d * p.max_pages + full] = page;
            p.refs[page] = 1;
        }
        p.lens[d] = m;
    }
    if (i == 0) p.scratch[kScrRefused] = 0;
}

// Fork, second half: block (x, i) copies its share of the (layer, K or V, head) runs of pair i's
// partly filled page, rows 0 .. rows % page_size.
__global__ void __launch_bounds__(256) pages_fork_copy_kernel(const PagesView p, const int *src, const int *dst) {
    pdl_launch_dependents();
    pdl_wait();
    if (p.scratch[kScrRefused]) return;
    const int s = src[blockIdx.y], d = dst[blockIdx.y];
    const int m = p.lens[d], full = m / p.page_size, tail = m % p.page_size;
    if (!tail) return;
    const int from = p.table[(size_t)s * p.max_pages + full], to = p.table[(size_t)d * p.max_pages + full];
    const int vr = p.row_bytes >> 4, words = tail * vr;  // 16-byte words a row, a run
    const int runs = 2 * p.n_layers * p.n_kv_heads;
    const int lane = threadIdx.x & 31, nw = gridDim.x * (blockDim.x >> 5);
    for (int u = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); u < runs; u += nw) {
        const int h = u % p.n_kv_heads, lv = u / p.n_kv_heads, l = lv >> 1;
        char *pool = (lv & 1 ? p.v : p.k) + l * p.layer_stride + h * p.head_stride;
        const char *a = pool + from * p.page_stride;
        char *b = pool + to * p.page_stride;
        copy_words<32, 4>(a, b, lane, words, vr, p.row_stride);
    }
}

// Free, and the plan of a compaction: after the counts have dropped, n_live pages are held;
// the k-th free page below n_live takes the k-th held page at or above it, so no page is both read
// and written and the moves can run in any order.
__global__ void __launch_bounds__(kT) pages_free_kernel(const PagesView p, int n, const int *seqs, int compact) {
    __shared__ int buf[64], sq[kPagesMaxCall], len_s[kPagesMaxCall], why;
    const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int s = i < n ? seqs[i] : -1;
    sq[i] = s;
    __syncthreads();
    bool bad = i < n && (s < 0 || s >= p.n_seqs);
    int m = 0;
    if (i < n && !bad) {
        bool again = false;  // a sequence named twice is freed once
        for (int j = 0; j < i; ++j) again |= sq[j] == s;
        m = again ? 0 : p.lens[s];
        bad = m < 0 || m > (long long)p.max_pages * p.page_size;
    }
    len_s[i] = bad ? 0 : ceil_div_d(m, p.page_size);
    if (i == 0) why = 0;
    if (__syncthreads_or(bad)) return refuse(p, L2_PAGES_ERR_ARGS);
    auto held = [&](auto take) {  // every page of the sequences
        for (int e = warp; e < n; e += kT / 32) {
            const int *t = p.table + (size_t)sq[e] * p.max_pages;
            for (int j = lane; j < len_s[e]; j += 32) take(t[j]);
        }
    };
    held([&](int page) {
        if (!page_ok(p, page))
            atomicOr(&why, L2_DEV_ERR_BOUNDS);
        else if (atomicSub(p.refs + page, 1) <= 0)  // no holder left
            atomicOr(&why, L2_PAGES_ERR_ARGS);
    });
    __syncthreads();
    if (why) {  // nothing changes: what was taken is put back
        held([&](int page) {
            if (page_ok(p, page)) atomicAdd(p.refs + page, 1);
        });
        return refuse(p, why);
    }
    if (i < n) p.lens[s] = 0;
    if (i == 0) p.scratch[kScrRefused] = 0;
    if (!compact) return;
    __syncthreads();
    int live = 0;
    for (int b = i; b < p.n_pages; b += kT) live += __ldcg(p.refs + b) > 0;  // past L1: the counts were changed by atomics
    int n_live;
    block_scan(live, &n_live, buf);
    int *hole = p.scratch + kScrHead, *mover = hole + p.n_pages, *to = mover + p.n_pages;
    int moved = 0;
    // holes below n_live ascending, then held pages from n_live on ascending: as many of one as of the other.  to: where each
    // page's rows will be, -1 for pages that nobody holds
    for (int pass = 0; pass < 2; ++pass) {
        int found = 0;
        const int lo = pass ? n_live : 0, hi = pass ? p.n_pages : n_live;
        for (int base = lo; base < hi; base += 4 * kT) {
            const int i0 = base + 4 * i;
            bool f[4];
            int c = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j] = i0 + j < hi && (__ldcg(p.refs + i0 + j) > 0) == (pass == 1);
                c += f[j];
            }
            int total;
            int at = found + block_scan(c, &total, buf);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + j < hi) {
                    to[i0 + j] = f[j] == (pass == 1) ? i0 + j : -1;
                    if (f[j]) (pass ? mover : hole)[at++] = i0 + j;
                }
            found += total;
        }
        moved = found;
    }
    __syncthreads();
    for (int e = i; e < moved; e += kT) {
        const int a = mover[e], b = hole[e];
        to[a] = b;
        p.refs[b] = __ldcg(p.refs + a);
        p.refs[a] = 0;
    }
    if (i == 0) p.scratch[kScrMoved] = moved;
}

// Compaction: the moved pages' rows in every layer, and the tables' entries.  A run is one page's
// rows of one (layer, K or V, head), or all its heads where they lie side by side (`heads` 1).  A word a thread at a time: more
// loads before the stores were slower (356 MB moved: 125 us, 134 with two, 149 with four), while a fork's copies, from rows that
// L2 holds, and an append's, whose rows come side by side, gain from four (63 children of 7B: 59 -> 57 us; 1.4 GB: 225 -> 219).
constexpr int kCompactThreads = 512;
__global__ void __launch_bounds__(kCompactThreads, 4) pages_compact_kernel(const PagesView p, int heads, int rows, int row_bytes) {
    pdl_launch_dependents();
    pdl_wait();
    if (p.scratch[kScrRefused]) return;
    const int moved = p.scratch[kScrMoved];
    const int *hole = p.scratch + kScrHead, *mover = hole + p.n_pages, *to = mover + p.n_pages;
    if (!moved) return;
    const int tid = blockIdx.x * blockDim.x + threadIdx.x, nt = gridDim.x * blockDim.x;
    for (long long e = tid; e < (long long)p.n_seqs * p.max_pages; e += nt) {
        const int s = (int)(e / p.max_pages), j = (int)(e - (long long)s * p.max_pages);
        const int m = p.lens[s];
        if (m <= 0 || j >= ceil_div_d(m, p.page_size)) continue;
        const int page = p.table[e], now = page_ok(p, page) ? to[page] : -1;
        if (now < 0)  // left as it is
            atomicOr(p.err, page_ok(p, page) ? L2_PAGES_ERR_ARGS : L2_DEV_ERR_BOUNDS);
        else if (now != page)
            p.table[e] = now;
    }
    const int vr = row_bytes >> 4, words = rows * vr;
    const long long units = (long long)moved * 2 * p.n_layers * heads;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int h = (int)(u % heads);
        const long long x = u / heads;
        const int lv = (int)(x % (2 * p.n_layers)), e = (int)(x / (2 * p.n_layers)), l = lv >> 1;
        char *pool = (lv & 1 ? p.v : p.k) + l * p.layer_stride + h * p.head_stride;
        const char *a = pool + mover[e] * p.page_stride;
        char *b = pool + hole[e] * p.page_stride;
        copy_words<kCompactThreads, 1>(a, b, threadIdx.x, words, vr, p.row_stride);
    }
}

namespace {

// Every kernel here is launched as a dependent of what is before it in the stream: its blocks come up while that
// ends, and wait for its end before they read anything.
cudaError_t launch(void *fn, dim3 grid, int threads, void **args, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_pages_extend(const PagesView &p, int n, const int *seqs, const int *starts, int rows, cudaStream_t s) {
    void *args[] = {const_cast<PagesView *>(&p), &n, &seqs, &starts, &rows};
    return launch(reinterpret_cast<void *>(pages_extend_kernel), dim3(1), kT, args, s);
}

cudaError_t launch_pages_rows(const PagesView &p, const PagesAppend &a, bool read, cudaStream_t s) {
    if (a.rows == 0) return cudaSuccess;
    int per = 4;
    void *args[] = {const_cast<PagesView *>(&p), const_cast<PagesAppend *>(&a), &per};
    const long long warps = (long long)a.rows * ((a.n_layers + per - 1) / per);
    return launch(read ? reinterpret_cast<void *>(pages_rows_kernel<true>) : reinterpret_cast<void *>(pages_rows_kernel<false>), dim3((unsigned)((warps + 7) / 8)), 256, args, s);
}

cudaError_t launch_pages_fork(const PagesView &p, int n, const int *src, const int *dst, const int *rows, cudaStream_t s) {
    void *args[] = {const_cast<PagesView *>(&p), &n, &src, &dst, &rows};
    cudaError_t e = launch(reinterpret_cast<void *>(pages_fork_kernel), dim3(1), kT, args, s);
    if (e != cudaSuccess) return e;
    const long long runs = 2ll * p.n_layers * p.n_kv_heads;
    long long gx = (runs + 31) / 32;  // about four runs a warp
    if (gx > 256) gx = 256;
    void *args2[] = {const_cast<PagesView *>(&p), &src, &dst};
    return launch(reinterpret_cast<void *>(pages_fork_copy_kernel), dim3((unsigned)gx, n), 256, args2, s);
}

cudaError_t launch_pages_free(const PagesView &p, int n, const int *seqs, bool compact, int num_sms, cudaStream_t s) {
    int c = compact ? 1 : 0;
    void *args[] = {const_cast<PagesView *>(&p), &n, &seqs, &c};
    cudaError_t e = launch(reinterpret_cast<void *>(pages_free_kernel), dim3(1), kT, args, s);
    if (e != cudaSuccess || !compact) return e;
    // heads and rows that lie side by side are one run
    int heads = p.n_kv_heads, rows = p.page_size, bytes = p.row_bytes;
    if (p.row_stride == (long long)p.row_bytes && p.head_stride == (long long)rows * bytes) {
        bytes *= rows * heads;
        rows = heads = 1;
    } else if (p.head_stride == (long long)p.row_bytes && p.row_stride == (long long)heads * bytes) {
        bytes *= rows * heads;
        rows = heads = 1;
    } else if (p.row_stride == (long long)p.row_bytes) {
        bytes *= rows;
        rows = 1;
    }
    void *args2[] = {const_cast<PagesView *>(&p), &heads, &rows, &bytes};
    return launch(reinterpret_cast<void *>(pages_compact_kernel), dim3(num_sms * 4), kCompactThreads, args2, s);
}

}  // namespace l2
