"""The paged cache on the GPU: bookkeeping and row movement equal to the plain
statement of tests/pages_ref.py, and attention against 64 bits.

Tolerance of attention, element by element (u = 2^-24, n keys, head size d):
a score is a sum of d products, each within 2^-21 of its value (fp32 caches:
tf32 halves; 16-bit caches: exact), added in fp32 by steps that may truncate
(2u each), so it is off by at most e = (2^-21 + 2 d u) * scale * sum|q k| plus
8u of its size for the scaling; a weight is then off by 2 (e + 8 u |x|) relative
(numerator and denominator), plus, in 16-bit caches, at most half a step of the
type where the tensor cores take it as a 16-bit value (the sum l is of the
unrounded weights, so the numerator alone is off); the sum over keys takes at most one add per 8 keys and three chained
products each, every one at most 2u of the sum of w |v|.  The output adds half
a step of its type.
"""
import math

import numpy as np
import pytest

from tests import pages_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24


def dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def make_pool(dtype, n_layers, n_pages, kv, ps, hs, n_seqs, max_pages, order="head", fill=None):
    """Pool tensors in one of two memory orders, filled with `fill` (default: seeded noise)."""
    shape = (n_layers, n_pages, kv, ps, hs) if order == "head" else (n_layers, n_pages, ps, kv, hs)
    g = torch.Generator(device="cuda").manual_seed(n_pages * 31 + ps)
    kv_t = []
    for _ in range(2):
        t = torch.randn(shape, generator=g, device="cuda").to(dtype) if fill is None else torch.full(shape, fill, dtype=dtype, device="cuda")
        kv_t.append(t if order == "head" else t.transpose(2, 3))
    return pkg.PagePool.from_tensors(kv_t[0], kv_t[1], dev(np.zeros(n_pages)), dev(np.zeros(n_seqs)),
                                     dev(np.zeros((n_seqs, max_pages))))


def same_books(pool, ref):
    assert pool.lens.cpu().numpy().tolist() == ref.lens.tolist()
    assert pool.refs.cpu().numpy().tolist() == ref.refs.tolist()
    t = pool.table.cpu().numpy()
    for s in range(len(ref.lens)):
        h = ref.held(s)
        assert t[s, :h].tolist() == ref.table[s, :h].tolist(), s


@pytest.mark.parametrize("dtype,ps,kv,hs,order", [("fp32", 16, 4, 8, "head"), ("bf16", 7, 3, 48, "row"),
                                                  ("fp16", 1, 2, 64, "head"), ("fp32", 32, 1, 128, "row"),
                                                  ("bf16", 128, 2, 8, "head")])
def test_random_histories_match_the_plain_statement(dtype, ps, kv, hs, order):
    rng = np.random.default_rng(ps * 100 + hs)
    L, n_pages, n_seqs, max_pages = 3, 90, 24, 12
    pool = make_pool(DT[dtype], L, n_pages, kv, ps, hs, n_seqs, max_pages, order)
    ref = pages_ref.RefPool(n_pages, ps, n_seqs, max_pages)
    k, v = pool.k.clone(), pool.v.clone()  # the expected rows, page by page
    refused = 0
    for step in range(60):
        op = rng.choice(["append", "append", "fork", "free", "compact"])
        if op == "append":
            seqs = rng.permutation(n_seqs)[:rng.integers(1, n_seqs)]
            counts = rng.integers(0, 2 * ps + 2, len(seqs)) if step % 3 else np.ones(len(seqs), int)
            counts = [int(c) for c in counts]
            before = [a.copy() for a in (ref.refs, ref.lens, ref.table)]
            places = ref.append(seqs, counts)
            rows = sum(counts)
            # new rows as part of a wider tensor (a fused projection's output)
            wide = torch.randn((L, rows, 3 * kv, hs), device="cuda").to(DT[dtype])
            nk, nv = wide[:, :, kv:2 * kv], wide[:, :, 2 * kv:]
            starts = None if all(c == 1 for c in counts) else dev(np.concatenate([[0], np.cumsum(counts)]))
            if step % 2:
                pool.append(nk, nv, dev(seqs), starts)
            else:  # one layer after the other
                for layer in range(L):
                    pool.append(nk[layer], nv[layer], dev(seqs), starts, layer=layer)
            if places is None:
                refused += 1
                ref.refs, ref.lens, ref.table = before
                with pytest.raises(pkg.L2Error):
                    pool.check()
            elif rows:
                pages, at = torch.tensor([p[0] for p in places]).cuda(), torch.tensor([p[1] for p in places]).cuda()
                k.permute(1, 3, 0, 2, 4)[pages, at] = nk.transpose(0, 1)
                v.permute(1, 3, 0, 2, 4)[pages, at] = nv.transpose(0, 1)
        elif op == "fork":
            empty = [s for s in range(n_seqs) if ref.lens[s] == 0]
            full = [s for s in range(n_seqs) if ref.lens[s] > 0]
            if not empty or not full:
                continue
            n = int(rng.integers(1, min(len(empty), 9) + 1))
            dst = rng.permutation(empty)[:n]
            src = rng.choice(full, n)
            rows = None if step % 2 else [int(rng.integers(0, ref.lens[s] + 1)) for s in src]
            copies = ref.fork(src, dst, rows)
            pool.fork(dev(src), dev(dst), None if rows is None else dev(rows))
            if copies is None:
                refused += 1
                with pytest.raises(pkg.L2Error):
                    pool.check()
            else:
                for a, b, t in copies:
                    k[:, b, :, :t], v[:, b, :, :t] = k[:, a, :, :t], v[:, a, :, :t]
        else:
            seqs = rng.permutation(n_seqs)[:rng.integers(0, 6)]
            seqs = np.concatenate([seqs, seqs[:1]])  # one named twice
            moves = ref.free(seqs, op == "compact")
            pool.free(dev(seqs), compact=op == "compact")
            for a, b in moves:
                k[:, b], v[:, b] = k[:, a].clone(), v[:, a].clone()
        same_books(pool, ref)
        assert torch.equal(pool.k, k) and torch.equal(pool.v, v), (step, op)
    pool.check()
    assert refused < 40


def test_refused_calls_change_nothing_and_say_why():
    pool = make_pool(torch.float32, 2, 6, 2, 4, 8, 5, 4)
    rows = lambda n: torch.randn((2, n, 2, 8), device="cuda")  # noqa: E731
    x = rows(13)
    pool.append(x, x, dev([0, 2]), dev([0, 6, 13]))
    pool.check()
    books = [t.clone() for t in (pool.refs, pool.lens, pool.table, pool.k, pool.v)]

    def refused(call, text):
        call()
        with pytest.raises(pkg.L2Error, match=text):
            pool.check()
        for a, b in zip(books, (pool.refs, pool.lens, pool.table, pool.k, pool.v)):
            assert torch.equal(a, b)

    one, two, nine = rows(1), rows(2), rows(9)
    refused(lambda: pool.append(two, two, dev([0, 0])), "index")                       # a sequence twice
    refused(lambda: pool.append(one, one, dev([5])), "index")                          # no such sequence
    refused(lambda: pool.append(one, one, dev([-1])), "index")
    refused(lambda: pool.append(two, two, dev([0]), dev([0, 1])), "index")             # starts do not cover the rows
    refused(lambda: pool.append(two, two, dev([0, 1]), dev([0, 3, 2])), "index")       # starts descend
    refused(lambda: pool.append(rows(11), rows(11), dev([0]), dev([0, 11])), "index")  # longer than a table
    refused(lambda: pool.append(nine, nine, dev([1]), dev([0, 9])), "free pages")
    # ... and the other layers of a refused step are not written either
    refused(lambda: (pool.append(nine[0], nine[0], dev([1]), dev([0, 9]), layer=0),
                     pool.append(nine[1], nine[1], dev([1]), dev([0, 9]), layer=1)), "free pages")
    refused(lambda: pool.fork(dev([0]), dev([2])), "index")                            # not empty
    refused(lambda: pool.fork(dev([0, 0]), dev([1, 1])), "index")
    refused(lambda: pool.fork(dev([1]), dev([1])), "index")
    refused(lambda: pool.fork(dev([0]), dev([1]), dev([7])), "index")                  # more rows than there are
    refused(lambda: pool.fork(dev([0, 0, 0]), dev([1, 3, 4])), "free pages")
    refused(lambda: pool.free(dev([0, 9])), "index")
    q = torch.randn((2, 4, 8), device="cuda")
    out = torch.full((2, 4, 8), 7.0, device="cuda")
    for bad in (dict(seqs=dev([0, 5])), dict(seqs=dev([0, 2]), group_starts=dev([0, 1]), prefix_lens=dev([2])),
                dict(seqs=dev([0, 2]), group_starts=dev([0, 2]), prefix_lens=dev([-1])),
                dict(seqs=dev([0, 2]), group_starts=dev([1, 2]), prefix_lens=dev([1]))):
        refused(lambda: pool.attention(q, 0, out=out, **bad), "index")
        assert bool((out == 7.0).all())
    pool.append(one, one, dev([1]))   # the pool still works
    pool.check()


def test_appending_into_a_page_another_sequence_holds_is_refused():
    pool = make_pool(torch.float32, 1, 8, 1, 4, 8, 3, 4)
    x = torch.randn((1, 6, 1, 8), device="cuda")
    pool.append(x, x, dev([0]), dev([0, 6]))
    pool.table[1] = pool.table[0]      # a caller's own sharing of a partly filled page
    pool.lens[1] = 6
    pool.refs[pool.table[0, :2].long()] += 1
    before = pool.k.clone()
    pool.append(x[:, :1], x[:, :1], dev([1]))
    with pytest.raises(pkg.L2Error, match="inconsistent"):
        pool.check()
    assert torch.equal(pool.k, before)


# -- attention --------------------------------------------------------------

def build(dtype, H, kv, hs, ps, groups, order="head", seed=0, layers=1, poison=float("nan"), slack=3):
    """A pool whose sequences (in groups of (prefix, [own rows, ...])) hold shuffled pages; everything no sequence
    holds is `poison`.  Returns pool, per-sequence rows in 64 bits, starts, prefixes."""
    rng = np.random.default_rng(seed)
    lens = [p + n for p, own in groups for n in own]
    up = lambda n: -(-n // ps)  # noqa: E731
    need = sum(up(n) for n in lens) + slack
    n_seqs, max_pages = len(lens), max(up(max(lens)), 1) + 1
    pool = make_pool(DT[dtype], layers, need, kv, ps, hs, n_seqs, max_pages, order, fill=poison)
    ids = list(rng.permutation(need))
    table = rng.integers(0, need, (n_seqs, max_pages)).astype(np.int32)  # entries past a sequence's end: anything
    k_rows, v_rows, b = [], [], 0
    layer = layers - 1
    for prefix, own in groups:
        first = b
        for n in own:
            total = prefix + n
            k = torch.from_numpy(rng.standard_normal((total, kv, hs)).astype(np.float32)).to(DT[dtype])
            v = torch.from_numpy(rng.standard_normal((total, kv, hs)).astype(np.float32)).to(DT[dtype])
            if b != first:
                k[:prefix], v[:prefix] = k_rows[first][:prefix], v_rows[first][:prefix]
            for j in range(up(total)):
                if b != first and (j + 1) * ps <= prefix:
                    table[b, j] = table[first, j]
                    continue
                table[b, j] = ids.pop()
                m = min(ps, total - j * ps)
                pool.k[layer, int(table[b, j]), :, :m] = k[j * ps:j * ps + m].transpose(0, 1).cuda()
                pool.v[layer, int(table[b, j]), :, :m] = v[j * ps:j * ps + m].transpose(0, 1).cuda()
            k_rows.append(k)
            v_rows.append(v)
            b += 1
    pool.table.copy_(dev(table))
    pool.lens.copy_(dev(lens))
    starts = np.concatenate([[0], np.cumsum([len(own) for _, own in groups])])
    return pool, [(k.double().numpy(), v.double().numpy()) for k, v in zip(k_rows, v_rows)], starts, [p for p, _ in groups]


def check_attention(got, lse, q, rows, dtype, scale, seqs=None):
    hs = q.shape[2]
    half = torch.finfo(DT[dtype]).eps / 2
    qd = q.double().cpu().numpy()
    got = got.double().cpu().numpy()
    worst = 0.0
    for b in range(q.shape[0]):
        k, v = rows[b if seqs is None else seqs[b]]
        want, want_lse, mag, spread = pages_ref.attention(qd[b], k, v, scale)
        n = len(k)
        e = (2.0 ** -21 + 2 * hs * U) * spread + 8 * U * spread
        rel = 2 * e + (0 if dtype == "fp32" else half) + (3 * (n / 8 + 1) + 64) * 2 * U
        tol = rel * mag + half * (np.abs(want) + rel * mag) + 1e-38 + (2.0 ** -25 if dtype == "fp16" else 0)
        err = np.abs(got[b] - want)
        assert (err <= tol).all(), (b, n, float((err / tol).max()))
        worst = max(worst, float((err / tol).max()) if n else 0.0)
        if n:
            assert np.abs(lse[b].cpu().numpy() - want_lse).max() <= 2 * e + (3 * n / 8 + 64) * 2 * U + 2.0 ** -22 * (np.abs(want_lse).max() + 1)
        else:
            assert (got[b] == 0).all() and bool((lse[b] == -math.inf).all())
    return worst


CASES = [
    # heads, kv, hs, page size, groups (prefix, own rows)
    (8, 4, 8, 16, [(100, [1, 20, 7, 3])]),
    (6, 4, 48, 24, [(65, [1, 2, 0, 40])]),                     # heads not a multiple of KV heads
    (12, 12, 64, 7, [(33, [5] * 5), (0, [1, 0, 64, 65]), (129, [1])]),
    (32, 4, 64, 32, [(257, [3, 100, 31, 32, 33, 0] * 3)]),
    (32, 32, 128, 64, [(130, [1, 17]), (64, [64, 128, 1])]),
    (8, 1, 128, 16, [(200, [9] * 9)]),
    (16, 16, 16, 1, [(5, [3, 0])]),                            # pages of one row
    (40, 1, 32, 128, [(300, [11, 0, 5, 128])]),                # more heads on a KV head than one tile of rows
    (4, 2, 128, 1000, [(1500, [700, 1]), (0, [0])]),           # pages longer than a tile; an empty sequence
    (3, 3, 24, 5, [(0, [1])]),
    (2, 2, 64, 16, [(4000, [500] * 20)]),
    # prefixes that serve many rows: runs of 320 pairs, of 17 to 64, several groups, odd heads, every kind of page
    (32, 4, 64, 16, [(1000, [5] * 40)]),
    (32, 8, 128, 256, [(700, [3] * 33), (129, [1] * 5), (128, [0, 0, 0, 0, 0, 0, 1])]),
    (6, 4, 48, 8, [(515, [2] * 20)]),
    (12, 12, 128, 32, [(2048, [1] * 17)]),
    (8, 1, 64, 128, [(256, [0] * 32), (4000, [7] * 33)]),
    (4, 4, 96, 64, [(900, [70] * 129)]),
    (16, 2, 8, 64, [(1300, [1] * 16)]),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_matches_64_bits(case, dtype):
    H, kv, hs, ps, groups = CASES[case]
    pool, rows, starts, prefix = build(dtype, H, kv, hs, ps, groups, order="head" if case % 2 else "row", seed=case, layers=1 + case % 2)
    B = len(rows)
    g = torch.Generator(device="cuda").manual_seed(case)
    wide = torch.randn((B, H + 2 * kv, hs), generator=g, device="cuda").to(DT[dtype])  # q inside a fused projection
    q = wide[:, :H] * 2
    scale = 1 / math.sqrt(hs)
    lse = torch.empty((B, H), device="cuda")
    layer = pool.n_layers - 1
    out = pool.attention(q, layer, group_starts=dev(starts), prefix_lens=dev(prefix), lse=lse)
    pool.check()
    check_attention(out, lse, q, rows, dtype, scale)
    # the same rows without sharing, in another order, into a strided output
    order = np.random.default_rng(case).permutation(B)
    big = torch.full((B, H + 1, hs), 5.0, device="cuda").to(DT[dtype])
    out2 = pool.attention(q[torch.from_numpy(order).cuda()], layer, seqs=dev(order), out=big[:, :H], lse=lse)
    check_attention(out2, lse, q[torch.from_numpy(order).cuda()], rows, dtype, scale, seqs=order)
    assert bool((big[:, H] == 5.0).all())
    # twice the same call: the same bits
    again = pool.attention(q, layer, group_starts=dev(starts), prefix_lens=dev(prefix))
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))
    pool.check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 4.0])
def test_any_scale(scale, dtype):
    pool, rows, starts, prefix = build(dtype, 4, 2, 64, 16, [(300, [9] * 20)], seed=12)
    q = torch.randn((20, 4, 64), device="cuda").to(DT[dtype])
    lse = torch.empty((20, 4), device="cuda")
    out = pool.attention(q, 0, group_starts=dev(starts), prefix_lens=dev(prefix), scale=scale, lse=lse)
    pool.check()
    check_attention(out, lse, q, rows, dtype, scale)


def test_a_prefix_longer_than_a_member_is_cut_and_rows_may_repeat():
    pool, rows, starts, prefix = build("bf16", 8, 2, 64, 16, [(50, [30, 4, 10])], seed=3)
    q = torch.randn((4, 8, 64), device="cuda").to(torch.bfloat16)
    lse = torch.empty((4, 8), device="cuda")
    seqs = [0, 1, 2, 1]
    out = pool.attention(q, 0, seqs=dev(seqs), group_starts=dev([0, 4]), prefix_lens=dev([50]), lse=lse)
    check_attention(out, lse, q, rows, "bf16", 1 / 8, seqs=seqs)
    # a prefix length past the shortest member: its rows end where the sequence does
    same, rows2, _, _ = build("bf16", 8, 2, 64, 16, [(50, [0, 0, 0, 0])], seed=4)
    out = same.attention(q, 0, group_starts=dev([0, 4]), prefix_lens=dev([10 ** 6]), lse=lse)
    check_attention(out, lse, q, rows2, "bf16", 1 / 8)
    # groups without rows
    out = same.attention(q, 0, group_starts=dev([0, 0, 4, 4]), prefix_lens=dev([9, 20, 7]), lse=lse)
    check_attention(out, lse, q, rows2, "bf16", 1 / 8)
    same.check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_infinities_and_nan_of_visible_rows_show_as_in_the_formula(dtype):
    pool, rows, starts, prefix = build(dtype, 2, 2, 64, 16, [(40, [5, 9])], seed=5)
    page = int(pool.table[1, 2])            # sequence 1's own page (positions 32..47)
    pool.v[0, page, 0, 12] = float("nan")   # position 44: only sequence 1, KV head 0
    pool.k[0, page, 1, 12] = float("nan")
    q = torch.randn((2, 2, 64), device="cuda").to(DT[dtype])
    out = pool.attention(q, 0, group_starts=dev(starts), prefix_lens=dev(prefix))
    assert bool(out[0].isfinite().all()) and bool(out[1].isnan().all())
    pool.check()


def test_a_bad_page_is_reported_and_reads_nothing():
    pool, rows, starts, prefix = build("fp32", 4, 2, 32, 8, [(16, [20, 3])], seed=6)
    q = torch.randn((2, 4, 32), device="cuda")
    good = pool.attention(q, 0)
    for bad in (-1, pool.n_pages, 2 ** 31 - 1):
        pool.table[0, 4] = bad
        out = pool.attention(q, 0)
        with pytest.raises(pkg.L2Error, match="outside the pool"):
            pool.check()
        assert torch.equal(out[1], good[1]) and bool(out[0].isfinite().all())


def test_offsets_past_32_bits():
    # 2 x 5.4 GB: pages past 2^32 bytes
    ps, kv, hs, n_pages = 16, 4, 128, 330_000
    pool = pkg.PagePool.from_tensors(torch.zeros((1, n_pages, kv, ps, hs), dtype=torch.bfloat16, device="cuda"),
                                     torch.zeros((1, n_pages, kv, ps, hs), dtype=torch.bfloat16, device="cuda"),
                                     dev(np.zeros(n_pages)), dev(np.zeros(3)), dev(np.zeros((3, 8))))
    pool.refs[:n_pages - 12] = 1             # the free pages are the last ones
    x = torch.randn((2, 1, 50, kv, hs), device="cuda").to(torch.bfloat16)
    pool.append(x[0], x[1], dev([0]), dev([0, 50]))
    pool.fork(dev([0]), dev([1]))
    q = torch.randn((2, 8, hs), device="cuda").to(torch.bfloat16)
    lse = torch.empty((2, 8), device="cuda")
    out = pool.attention(q, 0, seqs=dev([0, 1]), group_starts=dev([0, 2]), prefix_lens=dev([48]), lse=lse)
    pool.check()
    assert int(pool.table[0, 0]) == n_pages - 12
    rows = [(x[0, 0].double().cpu().numpy(), x[1, 0].double().cpu().numpy())] * 2
    check_attention(out, lse, q, rows, "bf16", 1 / math.sqrt(hs))
    pool.refs[:n_pages - 12] = 0
    pool.free(compact=True)                  # and back to the lowest pages
    out2 = pool.attention(q, 0, seqs=dev([0, 1]), group_starts=dev([0, 2]), prefix_lens=dev([48]))
    pool.check()
    assert torch.equal(out, out2) and int(pool.table[:2, :4].max()) == 4


def test_a_step_captured_into_a_graph_follows_the_lengths():
    """Append, attention and fork of a decode step in one graph, replayed while sequences grow."""
    pool, rows, starts, prefix = build("fp32", 8, 4, 64, 16, [(70, [1, 5, 9])], seed=7, poison=0.0, slack=40)
    pool.refs.copy_(dev(np.bincount(np.concatenate([pool.table.cpu().numpy()[s, :-(-int(n) // 16)] for s, n in enumerate(pool.lens.tolist())]),
                                    minlength=pool.n_pages)))
    seqs = dev([0, 1, 2])
    k, v, q = (torch.zeros((3, n, 64), device="cuda") for n in (4, 4, 8))
    gs, pl = dev(starts), dev(prefix)
    lse = torch.zeros((3, 8), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.append(k, v, seqs, layer=0)
        out = pool.attention(q, 0, group_starts=gs, prefix_lens=pl, lse=lse)
    rows = [list(r) for r in rows]
    for step in range(9):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for s in range(3):
            rows[s][0] = np.concatenate([rows[s][0], k[s:s + 1].double().cpu().numpy()])
            rows[s][1] = np.concatenate([rows[s][1], v[s:s + 1].double().cpu().numpy()])
        check_attention(out, lse, q, rows, "fp32", 1 / 8)
    pool.check()


def test_two_streams_at_once_and_a_chosen_stream():
    pool, rows, starts, prefix = build("fp16", 16, 2, 64, 32, [(700, [50] * 12)], seed=8)
    q = [torch.randn((12, 16, 64), device="cuda").to(torch.float16) for _ in range(2)]
    gs, pl = dev(starts), dev(prefix)
    want = [pool.attention(x, 0, group_starts=gs, prefix_lens=pl) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(pool.attention(q[i], 0, group_starts=gs, prefix_lens=pl, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_serving_loop_of_all_operators(dtype):
    """A prompt appended, forked to children, grown and attended step by step, children freed, the pool closed
    up and the rest attended again: rows as kept on the host, attention in 64 bits."""
    rng = np.random.default_rng(11)
    L, H, kv, hs, ps = 2, 8, 2, 64, 16
    pool = pkg.PagePool(L, 64, kv, ps, hs, 8, 12, dtype=DT[dtype])
    new = lambda n: (torch.randn((L, n, kv, hs), device="cuda").to(DT[dtype]), torch.randn((L, n, kv, hs), device="cuda").to(DT[dtype]))  # noqa: E731
    k, v = new(75)
    pool.append(k, v, dev([0]), dev([0, 75]))
    pool.fork(dev([0] * 5), dev([1, 2, 3, 4, 5]))
    hist = {s: [k, v] for s in range(6)}
    live = [0, 1, 2, 3, 4, 5]
    for step in range(40):
        if step == 20:
            pool.free(dev([0, 2, 3]), compact=True)   # the parent among them: its pages live on in the children
            live = [1, 4, 5]
        order = [int(s) for s in rng.permutation(live)]
        k, v = new(len(order))
        for layer in range(L):
            pool.append(k[layer], v[layer], dev(order), layer=layer)
        for i, s in enumerate(order):
            hist[s] = [torch.cat([hist[s][0], k[:, i:i + 1]], 1), torch.cat([hist[s][1], v[:, i:i + 1]], 1)]
        if step % 10 in (0, 9):
            layer = step % L
            q = torch.randn((len(order), H, hs), device="cuda").to(DT[dtype])
            lse = torch.empty((len(order), H), device="cuda")
            out = pool.attention(q, layer, seqs=dev(order), group_starts=dev([0, len(order)]), prefix_lens=dev([75]), lse=lse)
            rows = [(hist[s][0][layer].double().cpu().numpy(), hist[s][1][layer].double().cpu().numpy()) for s in order]
            check_attention(out, lse, q, rows, dtype, 1 / 8)
    pool.check()
    assert int((pool.refs > 0).sum()) == int(pool.refs.nonzero().max()) + 1 or step > 20
    pool.free(dev(live))
    assert int(pool.refs.abs().sum()) == 0


# -- large calls ------------------------------------------------------------

def wide_pool(dtype, n_seqs, kv, hs, ps, lens, prefix_of=None, seed=0, order="head"):
    """A pool filled in a few tensor operations: sequence s holds lens[s] rows in shuffled pages; with prefix_of[s] = (first, n)
    its first n // ps pages are sequence `first`'s.  Returns the pool and a function that gathers a sequence's rows in 64 bits."""
    rng = np.random.default_rng(seed)
    held = [-(-int(n) // ps) for n in lens]
    own_from = [0 if prefix_of is None or prefix_of[s][0] == s else prefix_of[s][1] // ps for s in range(n_seqs)]
    need = sum(h - o for h, o in zip(held, own_from))
    n_pages, max_pages = need + 5, max(held) + 1
    ids = rng.permutation(n_pages).astype(np.int32)
    table, at = np.full((n_seqs, max_pages), -7, np.int32), 0
    for s in range(n_seqs):
        table[s, own_from[s]:held[s]] = ids[at:at + held[s] - own_from[s]]
        at += held[s] - own_from[s]
    for s in range(n_seqs):
        if own_from[s]:
            table[s, :own_from[s]] = table[prefix_of[s][0], :own_from[s]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = [torch.randn((1, n_pages, kv, ps, hs) if order == "head" else (1, n_pages, ps, kv, hs), generator=g, device="cuda").to(DT[dtype])
         for _ in range(2)]
    t = t if order == "head" else [x.transpose(2, 3) for x in t]
    pool = pkg.PagePool.from_tensors(t[0], t[1], dev(np.bincount(np.concatenate([table[s, :held[s]] for s in range(n_seqs)]), minlength=n_pages)),
                                     dev(lens), dev(table))

    def rows(s):
        pages = pool.table[s, :held[s]].long()
        return [x[0, pages].transpose(1, 2).reshape(-1, kv, hs)[:int(lens[s])].double() for x in (pool.k, pool.v)]
    return pool, rows


def check_wide(out, lse, q, rows, dtype, scale, which):
    """check_attention's bounds for the rows `which`, the 64-bit attention on the GPU."""
    H, hs = q.shape[1:]
    half = torch.finfo(DT[dtype]).eps / 2
    for b in which:
        k, v = rows(b)
        n, kv = k.shape[:2]
        if n == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        kvh = torch.arange(H, device="cuda") * kv // H
        qd = q[b].double()
        x = scale * torch.einsum("thd,hd->ht", k[:, kvh], qd)
        spread = float((abs(scale) * torch.einsum("thd,hd->ht", k[:, kvh].abs(), qd.abs())).max())
        w = torch.softmax(x, 1)
        want, mag = torch.einsum("ht,thd->hd", w, v[:, kvh]), torch.einsum("ht,thd->hd", w, v[:, kvh].abs())
        e = (2.0 ** -21 + 2 * hs * U) * spread + 8 * U * spread
        rel = 2 * e + (0 if dtype == "fp32" else half) + (3 * (n / 8 + 1) + 64) * 2 * U
        tol = rel * mag + half * (want.abs() + rel * mag) + 1e-38 + (2.0 ** -25 if dtype == "fp16" else 0)
        err = (out[b].double() - want).abs()
        assert bool((err <= tol).all()), (b, n, float((err / tol).max()))
        want_lse = torch.logsumexp(x, 1)
        assert float((lse[b].double() - want_lse).abs().max()) <= 2 * e + (3 * n / 8 + 64) * 2 * U + 2.0 ** -22 * (float(want_lse.abs().max()) + 1)


# rows, group sizes, prefix, most own rows, heads, KV heads, head size, page size
WIDE = [
    (193, None, 0, 40, 4, 2, 64, 16),               # one source more than a block plans for itself
    (97, [1] * 96 + [1], 30, 40, 2, 1, 64, 16),
    (300, [20] * 10 + [1] * 100, 300, 30, 4, 2, 64, 16),
    (1024, [1024], 700, 9, 8, 2, 128, 128),
    (1024, [1] * 1024, 100, 50, 2, 2, 32, 8),
    (1024, [512, 0, 0, 512], 257, 3, 1, 1, 64, 20),  # pages that fit no tensor-core box
    (640, [64] * 10, 1000, 5, 5, 1, 96, 64),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_calls_of_many_rows_and_groups(case, dtype):
    B, groups, prefix, own, H, kv, hs, ps = WIDE[case]
    rng = np.random.default_rng(case)
    lens = (prefix if groups else 0) + rng.integers(0, own + 1, B)
    firsts = None if groups is None else np.repeat(np.concatenate([[0], np.cumsum(groups)[:-1]]), groups)
    pool, rows = wide_pool(dtype, B, kv, hs, ps, lens, None if groups is None else [(int(f), prefix // ps * ps) for f in firsts], seed=case)
    if groups is not None:  # what of the prefix lies in a partly filled page is each sequence's own copy
        for t in (pool.k, pool.v):
            tail = prefix % ps
            if tail:
                col = pool.table[:, prefix // ps].long()
                t[0, col, :, :tail] = t[0, col[torch.from_numpy(firsts).cuda()], :, :tail]
    q = torch.randn((B, H, hs), device="cuda").to(DT[dtype])
    lse = torch.empty((B, H), device="cuda")
    args = {} if groups is None else dict(group_starts=dev(np.concatenate([[0], np.cumsum(groups)])), prefix_lens=dev([prefix] * len(groups)))
    out = pool.attention(q, 0, lse=lse, **args)
    pool.check()
    check_wide(out, lse, q, rows, dtype, 1 / math.sqrt(hs), sorted({0, 1, B - 1, *rng.integers(0, B, 40).tolist()}))
    # every row agrees with the call that shares nothing to the bounds of both, here the type's own step of |v| < 6
    plain = pool.attention(q, 0)
    assert float((out.float() - plain.float()).abs().max()) <= 6 * 4 * max(torch.finfo(DT[dtype]).eps, 1e-4)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,members,H,kv,hs", [(200_000, 1, 1, 1, 128), (70_001, 3, 4, 2, 64), (131_072, 20, 1, 1, 64),
                                               (100_003, 150, 1, 1, 64), (40_000, 9, 32, 1, 128)])
def test_long_prefixes_of_few_heads(dtype, n, members, H, kv, hs):
    """One KV head over many keys: an item in as many parts as it may have, and merges of several rounds."""
    lens = [n + 3 * s % 7 for s in range(members)]
    pool, rows = wide_pool(dtype, members, kv, hs, 16, lens, [(0, n // 16 * 16)] * members, seed=n)
    q = torch.randn((members, H, hs), device="cuda").to(DT[dtype])
    lse = torch.empty((members, H), device="cuda")
    out = pool.attention(q, 0, group_starts=dev([0, members]), prefix_lens=dev([n // 16 * 16]), lse=lse)
    pool.check()
    check_wide(out, lse, q, rows, dtype, 1 / math.sqrt(hs), {0, members // 2, members - 1})


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("members", [1, 20, 200])
def test_many_small_weights_beside_a_large_one(dtype, members):
    """2^17 keys of weight 2^-25.5 beside one of 1 whose V is 0: the output is what the small ones leave."""
    n, hs = 1 << 17, 64
    lens = [n + 1 if s == 0 else n for s in range(members)]
    pool, rows = wide_pool(dtype, members, 1, hs, 128, lens, [(0, n)] * members, seed=1)
    low = -25.5 * math.log(2)
    pool.k.zero_()
    pool.k[..., 0] = low          # rounded to the type, as the check's rows are
    pool.v.fill_(1.0)
    at = [(int(pool.table[0, 5]), 77), (int(pool.table[0, n // 128]), 0)]
    for page, row in at:
        pool.k[0, page, :, row, 0] = 0.0
        pool.v[0, page, :, row] = 0.0
    q = torch.zeros((members, 1, hs), device="cuda", dtype=DT[dtype])
    q[..., 0] = 1.0
    lse = torch.empty((members, 1), device="cuda")
    out = pool.attention(q, 0, scale=1.0, group_starts=dev([0, members]), prefix_lens=dev([n]), lse=lse)
    pool.check()
    check_wide(out, lse, q, rows, dtype, 1.0, {0, members - 1})


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_scores_of_minus_infinity(dtype):
    """Keys whose score is -inf have weight 0, in a prefix of its first tiles too; a row of nothing else is 0 / 0."""
    members, n, hs = 24, 512, 64
    pool, rows = wide_pool(dtype, members, 1, hs, 32, [n + 5] * members, [(0, n)] * members, seed=2)
    q = torch.randn((members, 1, hs), device="cuda").to(DT[dtype])
    q[..., 3] = 1.0
    pages = pool.table[0, :10].long()
    pool.k[0, pages, :, :, 3] = -math.inf        # keys 0 .. 319
    own = pool.table[2, :n // 32 + 1].long()
    lse = torch.empty((members, 1), device="cuda")
    args = dict(group_starts=dev([0, members]), prefix_lens=dev([n]), lse=lse)
    out = pool.attention(q, 0, **args)
    pool.check()
    assert bool(out.isfinite().all())
    for b in (0, 2, members - 1):
        k, v = rows(b)
        check_wide(out, lse, q, lambda _: (k[320:], v[320:]), dtype, 1 / 8, [b])
    pool.k[0, own, :, :, 3] = -math.inf          # all of sequence 2 (and the whole prefix, but not the others' own rows)
    out = pool.attention(q, 0, **args)
    assert bool(out[2].isnan().all()) and bool(out[[0, 1, 3]].isfinite().all())
    pool.check()


def test_bookkeeping_of_the_largest_calls():
    """1024 sequences a call, pools of more pages than one round of the search takes."""
    rng = np.random.default_rng(5)
    n_seqs, n_pages, ps, max_pages = 2048, 20000, 2, 40
    pool = make_pool(torch.bfloat16, 1, n_pages, 1, ps, 8, n_seqs, max_pages, fill=0.0)
    ref = pages_ref.RefPool(n_pages, ps, n_seqs, max_pages)
    k = pool.k.clone()

    def append(seqs, counts):
        rows = int(sum(counts))
        x = torch.randn((1, rows, 1, 8), device="cuda").to(torch.bfloat16)
        places = ref.append(seqs, [int(c) for c in counts])
        pool.append(x, x, dev(seqs), dev(np.concatenate([[0], np.cumsum(counts)])))
        k[0, torch.tensor([p[0] for p in places]).cuda(), 0, torch.tensor([p[1] for p in places]).cuda()] = x[0, :, 0]

    append(rng.permutation(1024), rng.integers(0, 30, 1024))
    same_books(pool, ref)
    src = rng.choice(np.flatnonzero(ref.lens[:1024] > 0), 1024)
    for a, b, t in ref.fork(src, np.arange(1024, 2048)):
        k[:, b, :, :t] = k[:, a, :, :t]
    pool.fork(dev(src), dev(np.arange(1024, 2048)))
    same_books(pool, ref)
    assert torch.equal(pool.k, k)
    for compact in (False, True):
        gone = rng.permutation(n_seqs)[:700]
        for a, b in ref.free(gone, compact):
            k[:, b] = k[:, a].clone()
        pool.free(dev(gone), compact=compact)
        same_books(pool, ref)
        assert torch.equal(pool.k, k)
    append(rng.permutation(n_seqs)[:1024], np.ones(1024, int))
    same_books(pool, ref)
    pool.check()
    assert torch.equal(pool.k, k) and torch.equal(pool.v, k)


def test_two_graphs_of_one_pool_and_calls_between():
    pool, rows, starts, prefix = build("bf16", 8, 2, 64, 16, [(300, [5, 9, 30])], seed=9, poison=0.0, slack=30)
    pool.refs.copy_(dev(np.bincount(np.concatenate([pool.table.cpu().numpy()[s, :-(-int(n) // 16)] for s, n in enumerate(pool.lens.tolist())]),
                                    minlength=pool.n_pages)))
    gs, pl, seqs = dev(starts), dev(prefix), dev([0, 1, 2])
    q = [torch.randn((3, 8, 64), device="cuda").to(torch.bfloat16) for _ in range(3)]
    k = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    lse = [torch.zeros((3, 8), device="cuda") for _ in range(3)]
    step, look = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(step):
        pool.append(k, k, seqs, layer=0)
        out0 = pool.attention(q[0], 0, group_starts=gs, prefix_lens=pl, lse=lse[0])
    with torch.cuda.graph(look):
        out1 = pool.attention(q[1], 0, lse=lse[1])
    rows = [list(r) for r in rows]
    for _ in range(4):
        step.replay()
        look.replay()
        out2 = pool.attention(q[2], 0, group_starts=gs, prefix_lens=pl, lse=lse[2])
        torch.cuda.synchronize()
        for s in range(3):
            rows[s] = [np.concatenate([r, k[s:s + 1].double().cpu().numpy()]) for r in rows[s]]
        for o, x, l in ((out0, q[0], lse[0]), (out1, q[1], lse[1]), (out2, q[2], lse[2])):
            check_attention(o, l, x, rows, "bf16", 1 / 8)
    pool.check()


def test_arguments_the_host_refuses():
    pool, rows, starts, prefix = build("bf16", 4, 2, 64, 16, [(30, [5, 9])], seed=10)
    q = torch.randn((2, 4, 64), device="cuda").to(torch.bfloat16)
    k = torch.randn((2, 2, 64), device="cuda").to(torch.bfloat16)
    wide = torch.zeros(4096, device="cuda", dtype=torch.bfloat16)
    i2 = dev([0, 1])
    for call in (lambda: pool.attention(q.float(), 0), lambda: pool.attention(q[..., :56], 0), lambda: pool.attention(q[:, 0], 0),
                 lambda: pool.attention(q, 1), lambda: pool.attention(q, -1), lambda: pool.attention(q[:, :1], 0),
                 lambda: pool.attention(q, 0, scale=math.inf), lambda: pool.attention(q, 0, scale=math.nan),
                 lambda: pool.attention(q, 0, seqs=i2.long()), lambda: pool.attention(q, 0, seqs=dev([0, 1, 0])),
                 lambda: pool.attention(q, 0, group_starts=dev([0, 2])), lambda: pool.attention(q, 0, prefix_lens=dev([2])),
                 lambda: pool.attention(q, 0, group_starts=dev([0, 1, 1, 2]), prefix_lens=dev([1, 1, 1])),   # more groups than rows
                 lambda: pool.attention(q, 0, group_starts=dev([0]), prefix_lens=dev([])),
                 lambda: pool.attention(q, 0, out=wide[:512].view(1, 8, 64)), lambda: pool.attention(q, 0, lse=wide[:8]),
                 lambda: pool.attention(q, 0, out=wide.as_strided((2, 4, 64), (64, 64, 1))),                 # rows over one another
                 lambda: pool.attention(q, 0, out=wide.as_strided((2, 4, 64), (128, 64, 1))),
                 lambda: pool.attention(wide.as_strided((2, 4, 64), (300, 68, 1)), 0),                       # strides of no whole words
                 lambda: pool.attention(wide[1:513].view(2, 4, 64), 0),                                      # a base of no whole word
                 lambda: pool.attention(torch.zeros((3, 4, 64), device="cuda", dtype=torch.bfloat16), 0),    # more rows than sequences
                 lambda: pool.attention(q[:0], 0),
                 lambda: pool.append(k, k, i2[:1], layer=0), lambda: pool.append(k, k[:1], i2, layer=0),
                 lambda: pool.append(k, k, [0, 1], layer=0), lambda: pool.append(k[:0], k[:0], i2[:0], layer=0),
                 lambda: pool.append(k, k, i2, layer=1), lambda: pool.append(k, k, i2, starts=dev([0, 2]), layer=0),
                 lambda: pool.append(k, k, i2), lambda: pool.append(k[:, :1], k[:, :1], i2, layer=0),
                 lambda: pool.fork(i2, i2[:1]), lambda: pool.fork(i2[:0], i2[:0]), lambda: pool.fork(i2.cpu(), i2),
                 lambda: pool.fork(dev(np.arange(1025)), dev(np.arange(1025))), lambda: pool.free(i2.float())):
        with pytest.raises((ValueError, pkg.L2Error)):
            call()
    pool.check()
    # rows within heads are as good as heads within rows
    out = torch.empty((4, 2, 64), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    lse = torch.empty((2, 4), device="cuda")
    pool.attention(q, 0, out=out, lse=lse)
    check_attention(out, lse, q, rows, "bf16", 1 / 8)


# -- prefixes long enough for the tensor cores ------------------------------

# heads, KV heads, head size, page size, memory order, groups of (prefix, members), most own rows, scale
LONG = [
    (8, 1, 64, 16, "head", [(21000, 40)], 9, 0.125),                      # 320 pairs: a run of 256 and one of 64
    (4, 4, 128, 64, "row", [(20011, 17)], 3, -0.1),                       # 17 pairs, a prefix that ends inside a page
    (2, 1, 8, 8, "head", [(60000, 65), (30100, 9)], 5, 0.5),              # 130 pairs, 18 pairs
    (3, 1, 32, 128, "row", [(50000, 43)], 40, 0.2),                       # 129 pairs
    (12, 4, 48, 256, "head", [(9000, 43), (0, 3), (8999, 30), (7, 1)], 70, 0.15),
    (5, 2, 96, 32, "row", [(16385, 48)], 2, 0.1),                         # heads not a multiple of KV heads
    (16, 2, 128, 128, "head", [(12800, 16), (12800, 3), (25600, 2)], 300, 0.09),
    (64, 1, 64, 32, "head", [(30000, 1), (4096, 9)], 0, 0.125),           # rows without rows of their own; a row alone
    (6, 6, 64, 20, "head", [(5000, 90)], 4, 0.125),                       # pages that only fp32 can read by tensor core
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_long_prefixes_of_many_pairs(case, dtype):
    H, kv, hs, ps, order, groups, own, scale = LONG[case]
    rng = np.random.default_rng(case)
    sizes = [m for _, m in groups]
    B = sum(sizes)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    firsts, prefix = np.repeat(starts[:-1], sizes), np.repeat([p for p, _ in groups], sizes)
    lens = prefix + rng.integers(0, own + 1, B)
    pool, rows = wide_pool(dtype, B, kv, hs, ps, lens, [(int(f), int(p) // ps * ps) for f, p in zip(firsts, prefix)], seed=case, order=order)
    for t in (pool.k, pool.v):  # the rest of a prefix lies in each sequence's own page
        for b in range(B):
            tail, col = int(prefix[b]) % ps, int(prefix[b]) // ps
            if tail and firsts[b] != b:
                t[0, int(pool.table[b, col]), :, :tail] = t[0, int(pool.table[firsts[b], col]), :, :tail]
    q = torch.randn((B, H, hs), device="cuda").to(DT[dtype])
    lse = torch.empty((B, H), device="cuda")
    args = dict(group_starts=dev(starts), prefix_lens=dev([p for p, _ in groups]), scale=scale)
    out = pool.attention(q, 0, lse=lse, **args)
    pool.check()
    check_wide(out, lse, q, rows, dtype, scale, sorted({0, 1, B - 1, *rng.integers(0, B, 12).tolist()}))
    again = pool.attention(q, 0, **args)
    assert torch.equal(out, again)
    # a table entry outside the pool: reported, and its rows count as zeros
    page = int(lens[0] > ps) and int(pool.table[0, 1])
    pool.table[pool.table == page] = pool.n_pages + 5
    out = pool.attention(q, 0, **args)
    with pytest.raises(pkg.L2Error, match="outside the pool"):
        pool.check()
    assert bool(out.isfinite().all())
    pool.k[0, page], pool.v[0, page] = 0, 0
    pool.table[pool.table == pool.n_pages + 5] = page
    zeros = pool.attention(q, 0, **args)
    assert torch.equal(out, zeros)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("hs", [64, 128])
def test_infinite_scores_in_long_prefixes(dtype, hs):
    """-inf in K: weight 0, in whole tiles and single keys; NaN in K and in a query: their own rows alone."""
    members, n, H = 40, 20000, 4
    pool, rows = wide_pool(dtype, members, 1, hs, 64, [n + s % 3 for s in range(members)], [(0, n // 64 * 64)] * members, seed=3)
    q = torch.randn((members, H, hs), device="cuda").to(DT[dtype])
    q[..., 3] = q[..., 3].abs() + 0.5
    gone = torch.zeros(n + 3, dtype=torch.bool, device="cuda")
    gone[:512] = True
    gone[10_000:10_030:7] = True
    for j in range(n // 64):  # the shared pages
        hit = gone[64 * j:64 * j + 64]
        if bool(hit.any()):
            pool.k[0, int(pool.table[0, j]), 0, hit, 3] = -math.inf
    q[7, 2] = math.nan
    lse = torch.empty((members, H), device="cuda")
    args = dict(group_starts=dev([0, members]), prefix_lens=dev([n // 64 * 64]))
    out = pool.attention(q, 0, lse=lse, **args)
    pool.check()
    assert bool(out[7, 2].isnan().all()) and int(out.isnan().sum()) == hs

    def visible(b):
        k, v = rows(b)
        keep = ~gone[:len(k)]
        return k[keep], v[keep]
    q[7, 2], out[7, 2], lse[7, 2] = q[7, 1], out[7, 1], lse[7, 1]
    check_wide(out, lse, q, visible, dtype, 1 / math.sqrt(hs), [0, 7, 13, members - 1])
    pool.k[0, int(pool.table[0, 100]), 0, 5, 1] = math.nan
    out = pool.attention(q, 0, **args)
    assert bool(out.isnan().all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_long_prefixes_captured_and_on_two_streams(dtype):
    members, n, H, hs = 48, 16_384, 4, 128
    pool, rows = wide_pool(dtype, members, 1, hs, 64, [n + s % 50 for s in range(members)], [(0, n)] * members, seed=4)
    q = [torch.randn((members, H, hs), device="cuda").to(DT[dtype]) for _ in range(2)]
    args = dict(group_starts=dev([0, members]), prefix_lens=dev([n]))
    want = [pool.attention(x, 0, **args) for x in q]
    lse = torch.empty((members, H), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pool.attention(q[0], 0, lse=lse, **args)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        for i in range(2):
            got[i].append(pool.attention(q[i], 0, stream=streams[i], **args))
        torch.cuda.synchronize()
        assert torch.equal(out, want[0])
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
    check_wide(out, lse, q[0], rows, dtype, 1 / math.sqrt(hs), [0, 1, members - 1])
    pool.check()


# -- reading back, and a decoder's cache in pages -----------------------------

@pytest.mark.parametrize("dtype,ps,kv,hs,order", [("fp32", 16, 4, 8, "head"), ("bf16", 7, 3, 48, "row"), ("fp16", 32, 1, 128, "head")])
def test_rows_read_back_are_the_rows_appended(dtype, ps, kv, hs, order):
    L, lens = 5, [40, 1, 0, 77]
    pool = make_pool(DT[dtype], L, 30, kv, ps, hs, 4, 12, order)
    starts = dev(np.concatenate([[0], np.cumsum(lens)]))
    x = torch.randn((2, L, sum(lens), kv, hs), device="cuda").to(DT[dtype])
    pool.append(x[0], x[1], dev([3, 0, 2, 1]), starts)
    wide = torch.full((2, L, sum(lens), kv + 2, hs), 3.0, device="cuda").to(DT[dtype])
    pool.read(wide[0, :, :, 1:-1], wide[1, :, :, 1:-1], dev([3, 0, 2, 1]), starts)
    assert torch.equal(wide[:, :, :, 1:-1], x) and bool((wide[:, :, :, [0, -1]] == 3).all())
    # one layer, the first rows only, a sequence twice
    part = torch.zeros((2, 8, kv, hs), device="cuda").to(DT[dtype])
    pool.read(part[0], part[1], dev([1, 1]), dev([0, 5, 8]), layer=3)
    pool.check()
    assert torch.equal(part[:, :5], x[:, 3, 41:46]) and torch.equal(part[:, 5:], x[:, 3, 41:44])
    # rows past the end stay and are reported; so are bad indices
    part.fill_(7.0)
    pool.read(part[0], part[1], dev([0, 9]), dev([0, 4, 8]), layer=0)
    with pytest.raises(pkg.L2Error, match="index"):
        pool.check()
    assert torch.equal(part[:, :1], x[:, 0, 40:41]) and bool((part[:, 1:] == 7).all())
    for bad in (lambda: pool.read(x[0, 0, :1].expand(2, kv, hs), x[1, 0, :1].expand(2, kv, hs), dev([3]), dev([0, 2]), layer=0),
                lambda: pool.read(x[0], x[1], dev([3]), dev([0, 1, 2]))):
        with pytest.raises((ValueError, pkg.L2Error)):
            bad()


def test_a_prompt_prefilled_once_starts_other_slots():
    import synth
    wl = synth.WORKLOADS["gqa_small"]
    w = pkg.to_device(synth.make_weights(wl))
    dec = pkg.Decoder(wl.config_tuple(), w, max_batch=3)
    head = dec.dim // dec.n_heads
    toks = synth.token_stream(wl, 0, 60)
    pool = pkg.PagePool(dec.n_layers, 40, dec.n_kv_heads, 16, head, 4, 8)
    torch.cuda.synchronize()
    dec.prefill(toks[:50], slot=1)
    dec.kv_to_pages(pool, 2, slot=1)
    with torch.cuda.stream(dec.stream):
        pool.fork(dev([2]), dev([0]))
        pool.free(dev([2]), compact=True)
    dec.kv_from_pages(pool, 0, 50, slot=0)
    dec.kv_from_pages(pool, 0, 33, slot=2)
    dec.sync()
    pool.check()
    assert [dec.position(s) for s in range(3)] == [50, 50, 33]
    for layer in range(dec.n_layers):
        want = dec.kv_export(layer, slot=1)
        for got, n in ((dec.kv_export(layer, slot=0), 50), (dec.kv_export(layer, slot=2), 33)):
            assert all(np.array_equal(a, b[:n]) for a, b in zip(got, want))
    # the slots go on alike: a step from the copied rows, and the rest of the prompt from the shorter copy
    out = torch.empty((3, wl.vocab_size), device="cuda")
    dec.prefill(toks[33:50], pos0=33, slot=2)
    dec.forward_batch([toks[50]] * 3, [50] * 3, out)
    dec.sync()
    assert torch.equal(out[0], out[1])
    assert float((out[2] - out[1]).abs().max()) <= 1e-4 * float(out[1].abs().max())  # other chunks of the prompt: other sums
    # attention over the pages agrees with the rows the decoder exports
    q = torch.randn((1, dec.n_heads, head), device="cuda")
    lse = torch.empty((1, dec.n_heads), device="cuda")
    k, v = (a.reshape(50, dec.n_kv_heads, head).astype(np.float64) for a in [x[:50] for x in dec.kv_export(1, slot=1)])
    check_attention(pool.attention(q, 1, seqs=dev([0]), lse=lse), lse, q, [(k, v)], "fp32", 1 / math.sqrt(head))
    # refusals
    other = pkg.PagePool(dec.n_layers, 4, dec.n_kv_heads, 16, head, 2, 2, dtype=torch.bfloat16)
    fresh = pkg.Decoder(wl.config_tuple(), w)
    for call in (lambda: dec.kv_to_pages(other, 0), lambda: dec.kv_from_pages(other, 0, 5), lambda: dec.kv_from_pages(pool, 0, 0),
                 lambda: dec.kv_from_pages(pool, 0, wl.seq_len + 1), lambda: dec.kv_to_pages(pool, 0, slot=3), lambda: fresh.kv_to_pages(pool, 0)):
        with pytest.raises(pkg.L2Error):
            call()
    dec.kv_from_pages(pool, 3, 1, slot=0)  # an empty sequence: the device's finding
    dec.sync()
    with pytest.raises(pkg.L2Error, match="index"):
        pool.check()


@pytest.mark.parametrize("bits,code,words", [(1, pkg.L2_ETIMEOUT, ["wait ran out"]), (2, pkg.L2_EDEVICE, ["outside the pool"]),
                                             (12, pkg.L2_EDEVICE, ["index arrays", "free pages"])])
def test_every_status_bit_has_its_words(bits, code, words):
    pool = make_pool(torch.float32, 1, 2, 1, 4, 8, 1, 2)
    pool.status.fill_(bits)
    with pytest.raises(pkg.L2Error) as e:
        pool.check()
    assert e.value.code == code and all(w in str(e.value) for w in words)
    pool.check()  # cleared
