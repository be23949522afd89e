// Host side of the paged-cache entry points declared in include/l2.h: argument checks, the
// device the pool lives on, and the launches.  No call allocates, waits or keeps anything.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/l2.h"
#include "l2_check.h"
#include "l2_kernels.h"
#include "l2_pages.h"

using namespace l2;

namespace {

constexpr unsigned kReady = 0x50a6e500u;  // with the pool's device below

// Everything about a pool that the host can see.
int check_pool(const char *who, const L2Pages *p, int *device) {
    if (!p) return refuse(L2_EINVAL, "%s: NULL pool", who);
    if (p->dtype != L2_F32 && p->dtype != L2_BF16 && p->dtype != L2_F16)
        return refuse(L2_EINVAL, "%s: dtype %d is not L2_F32, L2_BF16 or L2_F16", who, p->dtype);
    if (p->n_layers < 1 || p->n_pages < 1 || p->n_kv_heads < 1 || p->page_size < 1 || p->head_size < 1 || p->n_seqs < 1 ||
        p->max_pages < 1)
        return refuse(L2_EINVAL, "%s: every size of the pool must be positive", who);
    const long long es = elt_size(p->dtype), rb = p->head_size * es;
    if (p->head_size > 128 || rb % 16)
        return refuse(L2_EINVAL, "%s: head_size %d must be at most 128 and a multiple of %lld", who, p->head_size, 16 / es);
    if ((long long)p->max_pages * p->page_size > 0x3fffffffll)
        return refuse(L2_EINVAL, "%s: max_pages * page_size exceeds 2^30 - 1 positions", who);
    if ((long long)p->page_size * p->n_kv_heads * rb > 0x3fffffffll || (long long)p->n_layers * p->n_kv_heads > 0xffffffll)
        return refuse(L2_EINVAL, "%s: page_size, n_kv_heads or n_layers too large", who);
    const long long st[4] = {p->layer_stride, p->page_stride, p->head_stride, p->row_stride};
    const int n[4] = {p->n_layers, p->n_pages, p->n_kv_heads, p->page_size};
    static const char *names[4] = {"layer_stride", "page_stride", "head_stride", "row_stride"};
    for (int i = 0; i < 4; ++i) {
        if (n[i] == 1) continue;  // never stepped
        if (st[i] * es % 16 || st[i] < p->head_size)
            return refuse(L2_EINVAL, "%s: %s %lld must be at least head_size and a multiple of 16 bytes", who, names[i], st[i]);
        if (st[i] > (1ll << 40)) return refuse(L2_EINVAL, "%s: %s %lld too large", who, names[i], st[i]);
    }
    if (!rows_apart(st, n, 4, p->head_size)) return refuse(L2_EINVAL, "%s: the strides give two rows the same memory", who);
    const void *const ptrs[7] = {p->k, p->v, p->refs, p->lens, p->table, p->status, p->scratch};
    static const char *const ptr_names[7] = {"k", "v", "refs", "lens", "table", "status", "scratch"};
    for (int i = 0; i < 7; ++i)
        if (!ptrs[i]) return refuse(L2_EINVAL, "%s: %s is NULL", who, ptr_names[i]);
    for (int i = 0; i < 7; ++i)
        if (int rc = check_ptr(who, ptr_names[i], ptrs[i], i < 2 ? 16 : 4, device)) return rc;
    if (*device > 0xff) return refuse(L2_EINVAL, "%s: device %d", who, *device);
    return L2_OK;
}

// A pool that l2_pages_init has checked: its device and the kernels' view of it.
int view_pool(const char *who, const L2Pages *p, PagesView *v, int *device) {
    if (!p) return refuse(L2_EINVAL, "%s: NULL pool", who);
    if ((p->ready & ~0xffu) != kReady) return refuse(L2_EINVAL, "%s: the pool needs l2_pages_init", who);
    *device = (int)(p->ready & 0xffu);
    const long long es = elt_size(p->dtype), rb = p->head_size * es;
    v->k = static_cast<char *>(p->k);
    v->v = static_cast<char *>(p->v);
    v->refs = p->refs;
    v->lens = p->lens;
    v->table = p->table;
    v->err = p->status;
    v->scratch = p->scratch;
    v->layer_stride = p->n_layers > 1 ? p->layer_stride * es : 0;
    v->page_stride = p->n_pages > 1 ? p->page_stride * es : rb;
    v->head_stride = p->n_kv_heads > 1 ? p->head_stride * es : rb;
    v->row_stride = p->page_size > 1 ? p->row_stride * es : rb;
    v->n_layers = p->n_layers;
    v->n_pages = p->n_pages;
    v->n_kv_heads = p->n_kv_heads;
    v->page_size = p->page_size;
    v->n_seqs = p->n_seqs;
    v->max_pages = p->max_pages;
    v->row_bytes = (int)rb;
    return L2_OK;
}

int check_count(const char *who, int n, int least) {
    if (n < least || n > kPagesMaxCall) return refuse(L2_EINVAL, "%s: n = %d outside %d..%d", who, n, least, kPagesMaxCall);
    return L2_OK;
}

int check_attn_shape(const char *who, const L2Pages *p, int B, int G, int n_heads) {
    if (B < 1 || B > kPagesMaxCall) return refuse(L2_EINVAL, "%s: B = %d outside 1..%d", who, B, kPagesMaxCall);
    if (G < 0 || G > B) return refuse(L2_EINVAL, "%s: G = %d outside 0..B", who, G);
    if (n_heads < p->n_kv_heads || n_heads > 1024)
        return refuse(L2_EINVAL, "%s: n_heads = %d outside n_kv_heads..1024", who, n_heads);
    return L2_OK;
}

// Append, or the other way.
int move_rows(const char *who, const L2Pages *pool, const L2PagesRows *a, bool read, void *cuda_stream) {
    PagesView v;
    int device = -1, rc = view_pool(who, pool, &v, &device);
    if (rc) return rc;
    if (!a) return refuse(L2_EINVAL, "%s: NULL rows", who);
    if ((rc = check_count(who, a->n, 1))) return rc;
    if (a->rows < 0 || (!a->starts && a->rows != a->n) || a->rows > 0xffffff)
        return refuse(L2_EINVAL, "%s: rows = %d (without starts it is n, at most 2^24 - 1)", who, a->rows);
    if (a->layer < -1 || a->layer >= pool->n_layers)
        return refuse(L2_EINVAL, "%s: layer %d outside -1..%d", who, a->layer, pool->n_layers - 1);
    PagesAppend w{};
    const int es = elt_size(pool->dtype);
    w.n_layers = a->layer < 0 ? pool->n_layers : 1;
    w.layer0 = a->layer < 0 ? 0 : a->layer;
    if ((rc = check_stride(who, "layer_stride", a->layer_stride, w.n_layers, es)) ||
        (rc = check_stride(who, "row_stride", a->row_stride, a->rows, es)) ||
        (rc = check_stride(who, "head_stride", a->head_stride, pool->n_kv_heads, es)))
        return rc;
    if (read && a->extend) return refuse(L2_EINVAL, "%s: reading does not extend", who);
    const long long st[3] = {a->layer_stride, a->row_stride, a->head_stride};
    const int counts[3] = {w.n_layers, a->rows, pool->n_kv_heads};
    if (read && !rows_apart(st, counts, 3, pool->head_size)) return refuse(L2_EINVAL, "%s: the rows overlap", who);
    if ((rc = check_ptr(who, "seqs", a->seqs, 4, &device)) || (a->starts && (rc = check_ptr(who, "starts", a->starts, 4, &device))) ||
        (a->rows && ((rc = check_ptr(who, "k", a->k, 16, &device)) || (rc = check_ptr(who, "v", a->v, 16, &device)))))
        return rc;
    if ((long long)a->rows * w.n_layers > 0x3fffffffll)  // warps of the copy are counted in 32 bits
        return refuse(L2_EINVAL, "%s: %d rows of %d layers in one call", who, a->rows, w.n_layers);
    DeviceGuard guard;
    if (!guard.enter(device)) return refuse(L2_ECUDA, "%s: cannot use device %d", who, device);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    w.k = static_cast<char *>(const_cast<void *>(a->k));
    w.v = static_cast<char *>(const_cast<void *>(a->v));
    w.layer_stride = a->layer_stride * es;
    w.row_stride = a->row_stride * es;
    w.head_stride = a->head_stride * es;
    w.seqs = a->seqs;
    w.starts = a->starts;
    w.n = a->n;
    w.rows = a->rows;
    w.extended = a->extend != 0;
    if (a->extend) {
        cudaError_t e = launch_pages_extend(v, a->n, a->seqs, a->starts, a->rows, s);
        if (e != cudaSuccess) return finish(who, e);
    }
    return finish(who, launch_pages_rows(v, w, read, s));
}

// What attention of either kind takes: the layer, rows of queries and outputs, the scale.
int attn_rows(const char *who, const L2Pages *pool, const PagesView &v, int layer, int B, int n_heads, double scale, const void *q, void *out,
              float *lse, long long q_row, long long q_head, long long out_row, long long out_head, PagesAttn *k) {
    int rc;
    if (layer < 0 || layer >= pool->n_layers) return refuse(L2_EINVAL, "%s: layer %d outside 0..%d", who, layer, pool->n_layers - 1);
    const float scale_log2 = (float)(scale * 1.4426950408889634);  // scores are fp32
    if (!std::isfinite(scale) || !std::isfinite(scale_log2)) return refuse(L2_EINVAL, "%s: scale must be finite, in fp32 too", who);
    const int es = elt_size(pool->dtype);
    if ((rc = check_stride(who, "q_row_stride", q_row, B, es)) || (rc = check_stride(who, "q_head_stride", q_head, n_heads, es)) ||
        (rc = check_stride(who, "out_row_stride", out_row, B, es)) || (rc = check_stride(who, "out_head_stride", out_head, n_heads, es)))
        return rc;
    const long long out_st[2] = {out_row, out_head};
    const int out_n[2] = {B, n_heads};
    if (!rows_apart(out_st, out_n, 2, pool->head_size)) return refuse(L2_EINVAL, "%s: output rows overlap", who);
    k->k = v.k + layer * v.layer_stride;
    k->v = v.v + layer * v.layer_stride;
    k->lens = v.lens;
    k->table = v.table;
    k->err = v.err;
    k->page_stride = v.page_stride;
    k->head_stride = v.head_stride;
    k->row_stride = v.row_stride;
    k->q = static_cast<const char *>(q);
    k->out = static_cast<char *>(out);
    k->lse = lse;
    k->q_row = q_row * es;
    k->q_head = q_head * es;
    k->o_row = out_row * es;
    k->o_head = out_head * es;
    k->B = B;
    k->n_heads = n_heads;
    k->n_kv_heads = v.n_kv_heads;
    k->head_size = pool->head_size;
    k->page_size = v.page_size;
    k->max_pages = v.max_pages;
    k->n_seqs = v.n_seqs;
    k->n_pages = v.n_pages;
    k->dtype = pool->dtype;
    k->page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (v.page_size == 1 << i) k->page_shift = i;
    k->scale_log2 = scale_log2;
    return L2_OK;
}

// Most that an item costs in the plan: as many keys as a table has room for, in tiles of 8 that cost 7 (a team's of 16: 41).
long long longest_item(const PagesView &v, bool tree) { return (((long long)v.max_pages * v.page_size + 7) / 8) * (tree ? 21 : 7) + 128; }

int attn_launch(const char *who, const PagesAttn &k, int device, void *ws, long long ws_bytes, void *cuda_stream) {
    DeviceGuard guard;
    if (!guard.enter(device)) return refuse(L2_ECUDA, "%s: cannot use device %d", who, device);
    const int sms = sm_count(device);
    if (!sms) return refuse(L2_ECUDA, "%s: cannot query device %d", who, device);
    const long long need = (long long)pages_attn_ws_bytes(k.B, k.G, k.n_heads, k.n_kv_heads, k.head_size, sms, k.tree);
    if (ws_bytes < need) return refuse(L2_EINVAL, "%s: workspace of %lld bytes, %lld needed", who, ws_bytes, need);
    return finish(who, launch_pages_attn(k, ws, sms, static_cast<cudaStream_t>(cuda_stream)));
}

}  // namespace

long long l2_pages_scratch_ints(int n_pages) { return n_pages < 1 ? L2_EINVAL : kScrHead + 3ll * n_pages; }

int l2_pages_init(L2Pages *pool) {
    int device = -1;
    const int rc = check_pool("l2_pages_init", pool, &device);
    if (rc == L2_OK) pool->ready = kReady | (unsigned)device;
    return rc;
}

int l2_pages_append(const L2Pages *pool, const L2PagesRows *rows, void *cuda_stream) {
    return move_rows("l2_pages_append", pool, rows, false, cuda_stream);
}

int l2_pages_read(const L2Pages *pool, const L2PagesRows *rows, void *cuda_stream) {
    return move_rows("l2_pages_read", pool, rows, true, cuda_stream);
}

int l2_pages_fork(const L2Pages *pool, int n, const int *src, const int *dst, const int *rows, void *cuda_stream) {
    const char *who = "l2_pages_fork";
    PagesView v;
    int device = -1, rc = view_pool(who, pool, &v, &device);
    if (rc || (rc = check_count(who, n, 1)) || (rc = check_ptr(who, "src", src, 4, &device)) ||
        (rc = check_ptr(who, "dst", dst, 4, &device)) || (rows && (rc = check_ptr(who, "rows", rows, 4, &device))))
        return rc;
    DeviceGuard guard;
    if (!guard.enter(device)) return refuse(L2_ECUDA, "%s: cannot use device %d", who, device);
    return finish(who, launch_pages_fork(v, n, src, dst, rows, static_cast<cudaStream_t>(cuda_stream)));
}

int l2_pages_free(const L2Pages *pool, int n, const int *seqs, int compact, void *cuda_stream) {
    const char *who = "l2_pages_free";
    PagesView v;
    int device = -1, rc = view_pool(who, pool, &v, &device);
    if (rc || (rc = check_count(who, n, 0)) || (n && (rc = check_ptr(who, "seqs", seqs, 4, &device)))) return rc;
    DeviceGuard guard;
    if (!guard.enter(device)) return refuse(L2_ECUDA, "%s: cannot use device %d", who, device);
    const int sms = sm_count(device);
    if (!sms) return refuse(L2_ECUDA, "%s: cannot query device %d", who, device);
    return finish(who, launch_pages_free(v, n, seqs, compact != 0, sms, static_cast<cudaStream_t>(cuda_stream)));
}

long long l2_pages_attention_ws(const L2Pages *pool, int B, int G, int n_heads) {
    const char *who = "l2_pages_attention_ws";
    PagesView v;
    int device = -1, rc = view_pool(who, pool, &v, &device);
    if (rc || (rc = check_attn_shape(who, pool, B, G, n_heads))) return rc;
    const int sms = sm_count(device);
    if (!sms) return refuse(L2_ECUDA, "%s: cannot query device %d", who, device);
    return (long long)pages_attn_ws_bytes(B, G, n_heads, pool->n_kv_heads, pool->head_size, sms, false);
}

int l2_pages_attention(const L2Pages *pool, const L2PagesAttention *a, void *ws, long long ws_bytes, void *cuda_stream) {
    const char *who = "l2_pages_attention";
    PagesView v;
    int device = -1, rc = view_pool(who, pool, &v, &device);
    if (rc) return rc;
    if (!a) return refuse(L2_EINVAL, "%s: NULL arguments", who);
    if ((rc = check_attn_shape(who, pool, a->B, a->G, a->n_heads))) return rc;
    PagesAttn k{};
    if ((rc = attn_rows(who, pool, v, a->layer, a->B, a->n_heads, a->scale, a->q, a->out, a->lse, a->q_row_stride, a->q_head_stride,
                        a->out_row_stride, a->out_head_stride, &k)))
        return rc;
    if (!a->seqs && a->B > pool->n_seqs) return refuse(L2_EINVAL, "%s: B = %d exceeds the pool's %d sequences", who, a->B, pool->n_seqs);
    if ((rc = check_ptr(who, "q", a->q, 16, &device)) || (rc = check_ptr(who, "out", a->out, 16, &device)) ||
        (a->lse && (rc = check_ptr(who, "lse", a->lse, 4, &device))) || (a->seqs && (rc = check_ptr(who, "seqs", a->seqs, 4, &device))) ||
        (a->G && ((rc = check_ptr(who, "group_starts", a->group_starts, 4, &device)) ||
                  (rc = check_ptr(who, "prefix_lens", a->prefix_lens, 4, &device)))) ||
        (rc = check_ptr(who, "workspace", ws, 256, &device)))
        return rc;
    k.seqs = a->seqs;
    k.group_starts = a->group_starts;
    k.prefix_lens = a->prefix_lens;
    k.G = a->G;
    // a bound of the plan's costs: own keys and prefixes
    const long long gq = (k.n_heads + k.n_kv_heads - 1) / k.n_kv_heads, items = 2ll * k.B * ((gq + 15) / 16 + 1) * k.n_kv_heads;
    k.wide = items * longest_item(v, false) > 1ll << 30;
    return attn_launch(who, k, device, ws, ws_bytes, cuda_stream);
}

long long l2_pages_tree_attention_ws(const L2Pages *pool, int n, int rows, int n_heads) {
    const char *who = "l2_pages_tree_attention_ws";
    PagesView v;
    int device = -1, rc = view_pool(who, pool, &v, &device);
    if (rc || (rc = check_count(who, n, 1)) || (rc = check_attn_shape(who, pool, rows, 0, n_heads))) return rc;
    const int sms = sm_count(device);
    if (!sms) return refuse(L2_ECUDA, "%s: cannot query device %d", who, device);
    return (long long)pages_attn_ws_bytes(rows, n, n_heads, pool->n_kv_heads, pool->head_size, sms, true);
}

int l2_pages_tree_attention(const L2Pages *pool, const L2PagesTreeAttention *a, void *ws, long long ws_bytes, void *cuda_stream) {
    const char *who = "l2_pages_tree_attention";
    PagesView v;
    int device = -1, rc = view_pool(who, pool, &v, &device);
    if (rc) return rc;
    if (!a) return refuse(L2_EINVAL, "%s: NULL arguments", who);
    if ((rc = check_count(who, a->n, 1)) || (rc = check_attn_shape(who, pool, a->rows, 0, a->n_heads))) return rc;
    PagesAttn k{};
    if ((rc = attn_rows(who, pool, v, a->layer, a->rows, a->n_heads, a->scale, a->q, a->out, a->lse, a->q_row_stride, a->q_head_stride,
                        a->out_row_stride, a->out_head_stride, &k)))
        return rc;
    if ((rc = check_ptr(who, "q", a->q, 16, &device)) || (rc = check_ptr(who, "out", a->out, 16, &device)) ||
        (a->lse && (rc = check_ptr(who, "lse", a->lse, 4, &device))) || (rc = check_ptr(who, "seqs", a->seqs, 4, &device)) ||
        (rc = check_ptr(who, "starts", a->starts, 4, &device)) || (a->parents && (rc = check_ptr(who, "parents", a->parents, 4, &device))) ||
        (rc = check_ptr(who, "workspace", ws, 256, &device)))
        return rc;
    k.tree = true;
    k.seqs = a->seqs;
    k.group_starts = a->starts;
    k.parents = a->parents;
    k.G = a->n;
    // as above: all rows' pairs in items of 16, one more for each sequence
    const long long gq = (k.n_heads + k.n_kv_heads - 1) / k.n_kv_heads, items = (k.B * gq / 16 + k.G) * k.n_kv_heads;
    k.wide = items * longest_item(v, true) > 1ll << 30;
    return attn_launch(who, k, device, ws, ws_bytes, cuda_stream);
}

namespace {

int accept_rows(const char *who, const L2Pages *pool, const L2PagesAccept *a, bool find, void *cuda_stream) {
    PagesView v;
    int device = -1, rc = view_pool(who, pool, &v, &device);
    if (rc) return rc;
    if (!a) return refuse(L2_EINVAL, "%s: NULL arguments", who);
    if ((rc = check_count(who, a->n, 1))) return rc;
    if (a->rows < 0 || a->rows > L2_TREE_NODES * kPagesMaxCall)
        return refuse(L2_EINVAL, "%s: rows = %d outside 0..%d", who, a->rows, L2_TREE_NODES * kPagesMaxCall);
    if ((rc = check_ptr(who, "seqs", a->seqs, 4, &device)) || (rc = check_ptr(who, "starts", a->starts, 4, &device)) ||
        (rc = check_ptr(who, "counts", a->counts, 4, &device)) || (a->rows && (rc = check_ptr(who, "path", a->path, 4, &device))))
        return rc;
    if (find && ((a->rows && ((rc = check_ptr(who, "tokens", a->tokens, 4, &device)) || (rc = check_ptr(who, "targets", a->targets, 4, &device)))) ||
                 (a->parents && (rc = check_ptr(who, "parents", a->parents, 4, &device))) ||
                 (a->next && (rc = check_ptr(who, "next", a->next, 4, &device)))))
        return rc;
    if (!find && (a->tokens || a->targets || a->parents || a->next))
        return refuse(L2_EINVAL, "%s: tokens, targets, parents and next are NULL where the path is given", who);
    DeviceGuard guard;
    if (!guard.enter(device)) return refuse(L2_ECUDA, "%s: cannot use device %d", who, device);
    PagesAccept k{};
    k.seqs = a->seqs;
    k.starts = a->starts;
    k.n = a->n;
    k.rows = a->rows;
    k.find = find;
    k.parents = a->parents;
    k.tokens = a->tokens;
    k.targets = a->targets;
    k.path = a->path;
    k.counts = a->counts;
    k.next = a->next;
    return finish(who, launch_pages_accept(v, k, static_cast<cudaStream_t>(cuda_stream)));
}

}  // namespace

int l2_pages_accept(const L2Pages *pool, const L2PagesAccept *a, void *cuda_stream) {
    return accept_rows("l2_pages_accept", pool, a, true, cuda_stream);
}

int l2_pages_keep(const L2Pages *pool, const L2PagesAccept *a, void *cuda_stream) {
    return accept_rows("l2_pages_keep", pool, a, false, cuda_stream);
}
