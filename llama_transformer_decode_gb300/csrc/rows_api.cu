// Host side of the entry points on rows that a caller's own layer code makes (include/l2.h): rotary positions, rules on logits.
// Argument checks, the device the rows live on, and the launches.  No call allocates, waits or keeps anything.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/l2.h"
#include "l2_check.h"
#include "l2_kernels.h"
#include "l2_pages.h"
#include "l2_rows.h"

using namespace l2;

static_assert(L2_TREE_NODES == kTreeNodes && L2_ROPE_MAX == 2 * kRopePairs, "the header's limits are the kernels'");

namespace {

constexpr unsigned kRopeReady = 0x5207e001u;
constexpr unsigned kRulesReady = 0x5201e500u;  // with the rules' device below
constexpr double kTwoPi = 6.283185307179586476925286766559;

// Rows of a tensor: what its bytes are.
struct Extent {
    const char *p;
    long long row, head;  // strides in bytes
    int rows, heads, width;  // width: bytes of a row of a head
    long long columns() const { return (heads - 1) * head + width; }  // from a row's first byte to its last one's end
    long long bytes() const { return (rows - 1) * row + columns(); }
};
// Whether two tensors of as many rows have no byte in common.  Exact where their rows are alike apart (parts of a projection's output,
// side by side in a row or in each head); others are taken for sharing some unless one lies behind the other.
bool apart(const Extent &a, const Extent &b) {
    if (a.p + a.bytes() <= b.p || b.p + b.bytes() <= a.p) return true;
    if (a.rows != b.rows || (a.rows > 1 && a.row != b.row)) return false;
    const long long d = b.p - a.p, row = a.rows > 1 ? a.row : 0;
    if (row >= a.columns() && row >= b.columns()) {  // columns of one matrix
        const long long c = (d % row + row) % row;
        if (c >= a.columns() && c + b.columns() <= row) return true;
    }
    // A head of b and one of a, x bytes apart in the same row, meet where some difference of rows makes x + r * row less than a head's width
    // either way.
    auto meet = [&](long long x) {
        const long long w = a.width, v = b.width;  // from a's head on, b's begins above -v and below w
        if (!row) return x > -v && x < w;
        const long long r = (w - 1 - x) / row - ((w - 1 - x) % row < 0);  // the most rows that leave it below w
        return r >= 1 - a.rows && x + (r < a.rows ? r : a.rows - 1) * row > -v;
    };
    if (a.heads < 2 || b.heads < 2 || a.head == b.head) {  // differences of heads are all that matters
        const long long head = a.heads > 1 ? a.head : b.head;
        for (int h = 1 - a.heads; h < b.heads; ++h)
            if (meet(d + h * head)) return false;
        return true;
    }
    for (int i = 0; i < a.heads; ++i)
        for (int j = 0; j < b.heads; ++j)
            if (meet(d + j * b.head - i * a.head)) return false;
    return true;
}

int check_dtype(const char *who, const char *name, int dtype) {
    if (dtype != L2_F32 && dtype != L2_BF16 && dtype != L2_F16)
        return refuse(L2_EINVAL, "%s: %s %d is not L2_F32, L2_BF16 or L2_F16", who, name, dtype);
    return L2_OK;
}

// Queries, or keys: checked, and as the kernel takes them; *width: the elements that one access may take, lowered as this side needs.
int rope_side(const char *who, bool keys, const L2RopePlan *plan, const L2RopeRows *a, RopeSide *s, int *width, int *device) {
    const char *name = keys ? "k" : "q";
    const void *x = keys ? a->k : a->q;
    void *y = keys ? a->k_out : a->q_out;
    const int heads = keys ? a->n_kv_heads : a->n_heads, es = elt_size(a->dtype);
    const long long st[4] = {keys ? a->k_row_stride : a->q_row_stride, keys ? a->k_head_stride : a->q_head_stride,
                             keys ? a->k_out_row_stride : a->q_out_row_stride, keys ? a->k_out_head_stride : a->q_out_head_stride};
    *s = RopeSide{};
    if (heads < 0 || heads > 1024) return refuse(L2_EINVAL, "%s: %d heads of %s outside 0..1024", who, heads, name);
    if (!heads && x) return refuse(L2_EINVAL, "%s: %s has no heads", who, name);
    if (!heads) return L2_OK;
    int rc;
    if ((rc = check_ptr(who, name, x, es, device)) || (rc = check_ptr(who, keys ? "k_out" : "q_out", y, es, device))) return rc;
    for (int i = 0; i < 4; ++i)
        if (st[i] < 0 || st[i] > (1ll << 40)) return refuse(L2_EINVAL, "%s: stride %lld of %s", who, st[i], name);
    const int out_n[2] = {a->rows, heads};
    if (!rows_apart(st + 2, out_n, 2, a->head_size)) return refuse(L2_EINVAL, "%s: rows of %s_out overlap", who, name);
    s->x = static_cast<const char *>(x);
    s->y = static_cast<char *>(y);
    s->x_row = st[0] * es;
    s->x_head = st[1] * es;
    s->y_row = st[2] * es;
    s->y_head = st[3] * es;
    s->heads = heads;
    const bool in_place = x == y && (a->rows < 2 || st[0] == st[2]) && (heads < 2 || st[1] == st[3]);
    s->tail = in_place ? 0 : a->head_size - plan->rot_dim;
    if (!in_place && !apart({s->x, s->x_row, s->x_head, a->rows, heads, a->head_size * es}, {s->y, s->y_row, s->y_head, a->rows, heads, a->head_size * es}))
        return refuse(L2_EINVAL, "%s: %s_out shares memory with %s (in place: the same address and strides)", who, name, name);
    const unsigned long long bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y) | (a->rows > 1 ? s->x_row | s->y_row : 0) |
                                    (heads > 1 ? s->x_head | s->y_head : 0);
    while (bits % (*width * es) || s->tail % *width) *width /= 2;
    return L2_OK;
}

}  // namespace

int l2_rope_freqs(int rot_dim, double base, int scaling, double factor, double original_len, double low, double high, double *freqs) {
    const char *who = "l2_rope_freqs";
    if (!freqs) return refuse(L2_EINVAL, "%s: freqs is NULL", who);
    if (rot_dim < 2 || rot_dim > L2_ROPE_MAX || rot_dim % 2) return refuse(L2_EINVAL, "%s: rot_dim %d is not even or outside 2..%d", who, rot_dim, L2_ROPE_MAX);
    if (!std::isfinite(base) || base <= 0) return refuse(L2_EINVAL, "%s: base must be positive and finite", who);
    if (scaling < L2_ROPE_PLAIN || scaling > L2_ROPE_BANDS) return refuse(L2_EINVAL, "%s: scaling %d", who, scaling);
    if (scaling != L2_ROPE_PLAIN && (!std::isfinite(factor) || factor <= 0)) return refuse(L2_EINVAL, "%s: factor must be positive and finite", who);
    if (scaling == L2_ROPE_BANDS && !(std::isfinite(original_len) && original_len > 0 && std::isfinite(low) && std::isfinite(high) && low < high))
        return refuse(L2_EINVAL, "%s: original_len must be positive and low below high, all finite", who);
    if (scaling == L2_ROPE_BASE && rot_dim > 2) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == L2_ROPE_LINEAR) f /= factor;
        if (scaling == L2_ROPE_BANDS) {
            double s = (original_len * f / kTwoPi - low) / (high - low);
            s = s < 0 ? 0 : s > 1 ? 1 : s;
            f *= s + (1 - s) / factor;
        }
        if (!std::isfinite(f)) return refuse(L2_EINVAL, "%s: frequency %d is not finite", who, i);
        freqs[i] = f;
    }
    return L2_OK;
}

int l2_rope_plan(L2RopePlan *plan, int rot_dim, int layout, const double *freqs, double amplitude) {
    const char *who = "l2_rope_plan";
    if (!plan || !freqs) return refuse(L2_EINVAL, "%s: NULL pointer", who);
    plan->ready = 0;
    if (rot_dim < 2 || rot_dim > L2_ROPE_MAX || rot_dim % 2) return refuse(L2_EINVAL, "%s: rot_dim %d is not even or outside 2..%d", who, rot_dim, L2_ROPE_MAX);
    if (layout != L2_ROPE_INTERLEAVED && layout != L2_ROPE_HALF) return refuse(L2_EINVAL, "%s: layout %d", who, layout);
    if (!std::isfinite((float)amplitude)) return refuse(L2_EINVAL, "%s: amplitude must be finite, in fp32 too", who);
    for (int i = 0; i < rot_dim / 2; ++i) {
        if (!std::isfinite(freqs[i])) return refuse(L2_EINVAL, "%s: frequency %d is not finite", who, i);
        // of the frequency's size, which keeps a slow pair's bits when it turns back, too; whole turns do nothing at whole positions
        double t = std::fabs(freqs[i]) / kTwoPi;
        t -= std::floor(t);
        const double x = std::nearbyint(std::ldexp(t, 64));
        const unsigned long long turns = x >= 18446744073709551616.0 ? 0 : (unsigned long long)x;
        plan->turns[i] = freqs[i] < 0 ? 0 - turns : turns;
    }
    plan->rot_dim = rot_dim;
    plan->layout = layout;
    plan->amplitude = (float)amplitude;
    plan->ready = kRopeReady;
    return L2_OK;
}

int l2_rope(const L2RopePlan *plan, const L2RopeRows *a, void *cuda_stream) {
    const char *who = "l2_rope";
    if (!plan || !a) return refuse(L2_EINVAL, "%s: NULL arguments", who);
    if (plan->ready != kRopeReady) return refuse(L2_EINVAL, "%s: the plan needs l2_rope_plan", who);
    int rc, device = -1;
    if ((rc = check_dtype(who, "dtype", a->dtype))) return rc;
    if (a->rows < 0 || a->rows > 0xffffff) return refuse(L2_EINVAL, "%s: rows = %d outside 0..2^24 - 1", who, a->rows);
    if (a->head_size < plan->rot_dim || a->head_size > L2_ROPE_MAX)
        return refuse(L2_EINVAL, "%s: head_size %d outside %d..%d", who, a->head_size, plan->rot_dim, L2_ROPE_MAX);
    RopeParams p{};
    const bool half = plan->layout == L2_ROPE_HALF;
    int width = 16 / elt_size(a->dtype);
    while ((half ? plan->rot_dim / 2 : plan->rot_dim) % width) width /= 2;
    if (!a->rows) return L2_OK;
    if ((rc = check_ptr(who, "positions", a->positions, 4, &device)) || (rc = rope_side(who, false, plan, a, &p.s[0], &width, &device)) ||
        (rc = rope_side(who, true, plan, a, &p.s[1], &width, &device)))
        return rc;
    const RopeSide &q = p.s[0], &k = p.s[1];
    if (!q.heads && !k.heads) return L2_OK;
    if (q.heads && k.heads) {
        const int w = a->head_size * elt_size(a->dtype);
        const Extent qx = {q.x, q.x_row, q.x_head, a->rows, q.heads, w}, qy = {q.y, q.y_row, q.y_head, a->rows, q.heads, w};
        const Extent kx = {k.x, k.x_row, k.x_head, a->rows, k.heads, w}, ky = {k.y, k.y_row, k.y_head, a->rows, k.heads, w};
        if (!apart(qy, ky) || !apart(qy, kx) || !apart(ky, qx)) return refuse(L2_EINVAL, "%s: what is written of q or k shares memory with the other", who);
    }
    DeviceGuard guard;
    if (!guard.enter(device)) return refuse(L2_ECUDA, "%s: cannot use device %d", who, device);
    const int sms = sm_count(device);
    if (!sms) return refuse(L2_ECUDA, "%s: cannot query device %d", who, device);
    p.positions = a->positions;
    p.rows = a->rows;
    p.rot = plan->rot_dim;
    p.amplitude = plan->amplitude;
    for (int i = 0; i < p.rot / 2; ++i) p.turns[i] = plan->turns[i];
    return finish(who, launch_rope(p, a->dtype, half, width, sms, static_cast<cudaStream_t>(cuda_stream)));
}

int l2_token_rules_init(L2TokenRules *r) {
    const char *who = "l2_token_rules_init";
    if (!r) return refuse(L2_EINVAL, "%s: NULL rules", who);
    r->ready = 0;
    if (r->n_seqs < 1) return refuse(L2_EINVAL, "%s: n_seqs = %d", who, r->n_seqs);
    if (r->vocab_size < 1 || r->vocab_size > 1 << 24) return refuse(L2_EINVAL, "%s: vocab_size %d outside 1..2^24", who, r->vocab_size);
    if (r->max_len < 0 || r->max_len > 0xffff00) return refuse(L2_EINVAL, "%s: max_len %d outside 0..2^24 - 256", who, r->max_len);
    if (r->n_bias < 0 || r->n_bias > 0x3fffffff) return refuse(L2_EINVAL, "%s: n_bias %d outside 0..2^30 - 1", who, r->n_bias);
    if (r->n_seqs > 1 && (r->history_stride < r->max_len || r->history_stride > (1ll << 40)))
        return refuse(L2_EINVAL, "%s: history_stride %lld is below max_len or too large", who, r->history_stride);
    int rc, device = -1;
    if ((r->max_len && (rc = check_ptr(who, "history", r->history, 4, &device))) || (rc = check_ptr(who, "lens", r->lens, 4, &device))) return rc;
    const void *const optional[5] = {r->counted_from, r->repetition, r->presence, r->frequency, r->status};
    static const char *const names[5] = {"counted_from", "repetition", "presence", "frequency", "status"};
    for (int i = 0; i < 5; ++i)
        if (optional[i] && (rc = check_ptr(who, names[i], optional[i], 4, &device))) return rc;
    if (r->n_bias && ((rc = check_ptr(who, "bias_starts", r->bias_starts, 4, &device)) || (rc = check_ptr(who, "bias_tokens", r->bias_tokens, 4, &device)) ||
                      (rc = check_ptr(who, "bias_values", r->bias_values, 4, &device))))
        return rc;
    if (device > 0xff) return refuse(L2_EINVAL, "%s: device %d", who, device);
    r->ready = kRulesReady | (unsigned)device;
    return L2_OK;
}

int l2_token_rules(const L2TokenRules *r, const L2TokenRows *a, void *cuda_stream) {
    const char *who = "l2_token_rules";
    if (!r || !a) return refuse(L2_EINVAL, "%s: NULL arguments", who);
    if ((r->ready & ~0xffu) != kRulesReady) return refuse(L2_EINVAL, "%s: the rules need l2_token_rules_init", who);
    int rc, device = (int)(r->ready & 0xffu);
    if (a->n < 1 || a->n > 65535) return refuse(L2_EINVAL, "%s: n = %d outside 1..65535", who, a->n);
    if (a->rows < 0 || a->rows > 65535 || (!a->starts && a->rows != a->n))
        return refuse(L2_EINVAL, "%s: rows = %d outside 0..65535 (without starts it is n)", who, a->rows);
    if (!a->seqs && a->n > r->n_seqs) return refuse(L2_EINVAL, "%s: n = %d exceeds the rules' %d sequences", who, a->n, r->n_seqs);
    if ((rc = check_dtype(who, "dtype", a->dtype))) return rc;
    if (a->out_dtype != L2_F32 && a->out_dtype != a->dtype) return refuse(L2_EINVAL, "%s: out_dtype %d is neither L2_F32 nor the logits' type", who, a->out_dtype);
    const int es = elt_size(a->dtype), os = elt_size(a->out_dtype), V = r->vocab_size;
    const long long words = (V + 31) / 32;
    if (a->rows > 1 && (a->row_stride < 0 || a->row_stride > (1ll << 40))) return refuse(L2_EINVAL, "%s: row_stride %lld", who, a->row_stride);
    if (a->rows > 1 && (a->out_row_stride < V || a->out_row_stride > (1ll << 40)))
        return refuse(L2_EINVAL, "%s: out_row_stride %lld is below vocab_size or too large", who, a->out_row_stride);
    if (a->masks) {
        if (a->n_masks < 1 || (!a->mask_rows && a->n_masks < a->rows))
            return refuse(L2_EINVAL, "%s: n_masks = %d (without mask_rows there is one for each row)", who, a->n_masks);
        if (a->n_masks > 1 && (a->mask_stride < words || a->mask_stride > (1ll << 40)))
            return refuse(L2_EINVAL, "%s: mask_stride %lld is below a mask's %lld words or too large", who, a->mask_stride, words);
    }
    if (!a->rows) return L2_OK;
    if ((rc = check_ptr(who, "logits", a->logits, es, &device)) || (rc = check_ptr(who, "out", a->out, os, &device)) ||
        (a->seqs && (rc = check_ptr(who, "seqs", a->seqs, 4, &device))) || (a->starts && (rc = check_ptr(who, "starts", a->starts, 4, &device))) ||
        (a->parents && (rc = check_ptr(who, "parents", a->parents, 4, &device))) ||
        (a->drafted && (rc = check_ptr(who, "drafted", a->drafted, 4, &device))) || (a->masks && (rc = check_ptr(who, "masks", a->masks, 4, &device))) ||
        (a->masks && a->mask_rows && (rc = check_ptr(who, "mask_rows", a->mask_rows, 4, &device))))
        return rc;
    const bool in_place = a->out == a->logits && os == es && (a->rows < 2 || a->row_stride == a->out_row_stride);
    if (!in_place && !apart({static_cast<const char *>(a->logits), a->row_stride * es, 0, a->rows, 1, V * es},
                            {static_cast<const char *>(a->out), a->out_row_stride * os, 0, a->rows, 1, V * os}))
        return refuse(L2_EINVAL, "%s: out shares memory with the logits (in place: the same address, type and stride)", who);
    DeviceGuard guard;
    if (!guard.enter(device)) return refuse(L2_ECUDA, "%s: cannot use device %d", who, device);
    const int sms = sm_count(device);
    if (!sms) return refuse(L2_ECUDA, "%s: cannot query device %d", who, device);
    RulesParams p{};
    p.logits = static_cast<const char *>(a->logits);
    p.out = static_cast<char *>(a->out);
    p.in_row = a->row_stride * es;
    p.out_row = a->out_row_stride * os;
    p.seqs = a->seqs;
    p.starts = a->starts;
    p.parents = a->parents;
    p.drafted = a->drafted;
    p.history = r->history;
    p.lens = r->lens;
    p.counted = r->counted_from;
    p.repetition = r->repetition;
    p.presence = r->presence;
    p.frequency = r->frequency;
    p.bias_starts = r->bias_starts;
    p.bias_tokens = r->bias_tokens;
    p.bias_values = r->bias_values;
    p.masks = a->masks;
    p.mask_rows = a->masks ? a->mask_rows : nullptr;
    p.err = r->status;
    p.history_stride = r->history_stride;
    p.mask_stride = a->mask_stride;
    p.vocab = V;
    p.rows = a->rows;
    p.n = a->n;
    p.n_seqs = r->n_seqs;
    p.max_len = r->max_len;
    p.n_bias = r->n_bias;
    p.n_masks = a->n_masks;
    // elements an access, where every row begins on one: 8 bytes read and 16 written, or 16 of each (32 bytes written by a thread would be two
    // accesses that each leave every other sector half written)
    int vec = os == 2 ? 8 : 4;
    auto fits = [&](int w) {
        return !(reinterpret_cast<uintptr_t>(a->logits) % (w * es)) && !(reinterpret_cast<uintptr_t>(a->out) % (w * os)) &&
               (a->rows < 2 || (a->row_stride % w == 0 && a->out_row_stride % w == 0));
    };
    if (!fits(vec)) vec = fits(4) ? 4 : 1;
    return finish(who, launch_rules(p, a->dtype, a->out_dtype == L2_F32, vec, sms, static_cast<cudaStream_t>(cuda_stream)));
}
