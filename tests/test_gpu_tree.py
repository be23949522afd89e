"""Trees of drafted tokens over a page pool on the GPU: attention against 64 bits with the
tolerance of tests/test_gpu_pages.py (a token's keys are the committed rows and its path), acceptance equal to the
plain statement."""
import math

import numpy as np
import pytest

from tests import pages_ref, tree_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402
from tests.test_gpu_pages import DT, build, check_attention, dev, make_pool  # noqa: E402

F32 = torch.float32


def trees_of(kind, sizes, seed):
    rng = np.random.default_rng(seed)
    if kind == "chain":
        return [tree_ref.chain(n) for n in sizes]
    return [tree_ref.random_tree(rng, n, back={"wide": None, "deep": 3}.get(kind), roots=3 if kind == "forest" else 1) for n in sizes]


def rows_seen(rows, order, trees):
    """For each drafted token the rows (k, v) that it attends to."""
    got = []
    for s, parents in zip(order, trees):
        k, v = rows[s]
        base = len(k) - len(parents)
        for u in range(len(parents)):
            at = list(range(base)) + [base + j for j in tree_ref.line(parents, u)]
            got.append((k[at], v[at]))
    return got


def call_of(order, trees):
    starts = np.concatenate([[0], np.cumsum([len(t) for t in trees])])
    return dev(order), dev(starts), dev(np.concatenate([np.array(t, int) for t in trees])), int(starts[-1])


CASES = [
    # heads, kv, hs, page size, (committed rows, drafted) of each sequence, trees
    (8, 4, 8, 16, [(100, 7)], "wide"),
    (6, 4, 48, 24, [(65, 5), (0, 9), (1, 1), (300, 16)], "deep"),              # heads not a multiple of KV heads; nothing committed
    (12, 12, 64, 7, [(33, 16), (500, 3), (129, 1), (64, 33)], "forest"),       # several tokens without a parent
    (32, 4, 64, 32, [(257, 64), (1, 64), (999, 2)], "wide"),                   # the largest trees: 512 pairs of a KV head
    (32, 32, 128, 64, [(130, 64), (64, 20), (63, 1)], "chain"),
    (8, 1, 128, 16, [(200, 9), (0, 1), (17, 60)], "wide"),
    (16, 16, 16, 1, [(5, 12), (40, 4)], "deep"),                               # pages of one row
    (40, 1, 32, 128, [(300, 11), (128, 64)], "deep"),                          # 2560 pairs of one KV head
    (4, 2, 128, 1000, [(1500, 40), (999, 2)], "wide"),                         # pages longer than a tile
    (3, 3, 24, 5, [(0, 1)], "chain"),
    # committed rows long enough for the tensor cores
    (32, 4, 64, 16, [(4000, 40), (3500, 61), (700, 64), (4100, 1)], "wide"),
    (32, 8, 128, 256, [(5000, 33), (129, 5), (2048, 64)], "deep"),
    (12, 12, 128, 32, [(4096, 64), (4095, 63)], "wide"),
    (8, 1, 64, 128, [(9000, 64)], "chain"),
    (4, 4, 96, 64, [(6000, 64)] * 4, "deep"),
    (32, 32, 128, 16, [(1000, 24)] * 12, "wide"),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tree_attention_matches_64_bits(case, dtype):
    H, kv, hs, ps, seqs, kind = CASES[case]
    pool, rows, _, _ = build(dtype, H, kv, hs, ps, [(0, [p + n]) for p, n in seqs], order="head" if case % 2 else "row", seed=case,
                             layers=1 + case % 2)
    order = np.random.default_rng(case).permutation(len(seqs))
    trees = trees_of(kind, [seqs[s][1] for s in order], case)
    index, starts, parents, B = call_of(order, trees)
    g = torch.Generator(device="cuda").manual_seed(case)
    q = (torch.randn((B, H + 2 * kv, hs), generator=g, device="cuda").to(DT[dtype]))[:, :H] * 2   # inside a fused projection
    scale, layer = 1 / math.sqrt(hs), pool.n_layers - 1
    lse = torch.empty((B, H), device="cuda")
    big = torch.full((B + 2, H + 1, hs), 5.0, device="cuda").to(DT[dtype])   # a strided output with room around it
    out = pool.tree_attention(q, layer, index, starts, parents=parents, lse=lse, out=big[1:B + 1, :H])
    pool.check()
    check_attention(out, lse, q, rows_seen(rows, order, trees), dtype, scale)
    assert bool((big[:, H] == 5.0).all()) and bool((big[0] == 5.0).all()) and bool((big[B + 1] == 5.0).all())
    again = pool.tree_attention(q, layer, index, starts, parents=parents)
    assert torch.equal(out.contiguous().view(torch.uint8), again.view(torch.uint8))
    if kind == "chain":   # without parents: the same
        again = pool.tree_attention(q, layer, index, starts)
        assert torch.equal(out.contiguous().view(torch.uint8), again.view(torch.uint8))
    pool.check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,H,kv,hs", [(200, 8, 8, 64), (300, 4, 2, 16), (1000, 2, 1, 32)])
def test_many_small_trees(n, H, kv, hs, dtype):
    """More sequences than a block plans for itself, trees of none to five tokens, rows behind the last tree."""
    rng = np.random.default_rng(n)
    sizes = rng.integers(0, 1024 // n + 1, n)
    pool, rows, _, _ = build(dtype, H, kv, hs, 16, [(0, [int(c) + int(m)]) for c, m in zip(rng.integers(0, 60, n), sizes)], seed=n)
    order = rng.permutation(n)
    trees = trees_of("wide", [int(sizes[s]) for s in order], n)
    index, starts, parents, B = call_of(order, trees)
    room = min(1024, B + 10)
    parents = torch.cat([parents, torch.full((room - B,), 10 ** 6, dtype=torch.int32, device="cuda")])   # nobody's: not looked at
    q = torch.randn((room, H, hs), device="cuda").to(DT[dtype])
    out = torch.full((room, H, hs), 7.0, device="cuda").to(DT[dtype])
    lse = torch.full((room, H), 7.0, device="cuda")
    pool.tree_attention(q, 0, index, starts, parents=parents, out=out, lse=lse)
    pool.check()
    check_attention(out[:B], lse[:B], q[:B], rows_seen(rows, order, trees), dtype, 1 / math.sqrt(hs))
    assert bool((out[B:] == 7.0).all()) and bool((lse[B:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_trees_of_one_token_are_a_decode_step(dtype):
    pool, rows, _, _ = build(dtype, 8, 2, 64, 16, [(0, [n]) for n in (1, 2, 50, 700)], seed=3)
    q = torch.randn((4, 8, 64), device="cuda").to(DT[dtype])
    lse, want_lse = torch.empty((4, 8), device="cuda"), torch.empty((4, 8), device="cuda")
    out = pool.tree_attention(q, 0, dev(range(4)), dev(range(5)), lse=lse)
    want = pool.attention(q, 0, lse=want_lse)
    pool.check()
    # the same sums, cut among the walkers at other places: both within the bound of the same rows
    check_attention(out, lse, q, rows, dtype, 1 / 8)
    check_attention(want, want_lse, q, rows, dtype, 1 / 8)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,H,kv,hs,base", [("fp32", 4, 4, 64, 20), ("fp32", 32, 4, 64, 37), ("fp32", 8, 1, 128, 3), ("fp32", 2, 2, 16, 70),
                                                ("bf16", 4, 4, 64, 20), ("bf16", 32, 4, 64, 5000), ("bf16", 8, 1, 128, 3),
                                                ("fp16", 12, 2, 48, 33), ("fp16", 32, 8, 128, 4000), ("fp32", 32, 4, 128, 4000)])
def test_what_a_token_does_not_see_has_no_part_in_it(dtype, H, kv, hs, base, value):
    """Infinities and NaN in K and V of some drafted tokens: tokens that do not see them have the results they have without, and those that
    see them in V the formula's."""
    N = 40
    pool, rows, _, _ = build(dtype, H, kv, hs, 16, [(0, [base + N])], seed=base)
    trees = trees_of("wide", [N], 5)
    index, starts, parents, B = call_of([0], trees)
    q = torch.randn((B, H, hs), device="cuda").to(DT[dtype])
    scale = 1 / math.sqrt(hs)
    clean = pool.tree_attention(q, 0, index, starts, parents=parents)
    lse = torch.empty((B, H), device="cuda")

    def place(j):
        t = base + j
        return int(pool.table[0, t // 16]), t % 16
    in_k, in_v = (N - 1, 17), (N - 2, 9)
    for j in in_k:
        page, at = place(j)
        pool.k[0, page, :, at, 3] = value
    for j in in_v:
        page, at = place(j)
        pool.v[0, page, :, at, 5] = value
        pool.v[0, page, kv - 1, at, hs - 1] = value
    out = pool.tree_attention(q, 0, index, starts, parents=parents, lse=lse)
    pool.check()
    lines = [set(tree_ref.line(trees[0], u)) for u in range(N)]
    fine = [u for u in range(N) if not lines[u] & set(in_k + in_v)]
    assert 10 < len(fine) < N
    assert torch.equal(out[fine].view(torch.uint8), clean[fine].view(torch.uint8))
    check_attention(out[fine], lse[fine], q[fine], [rows_seen(rows, [0], trees)[u] for u in fine], dtype, scale)
    for u in range(N):
        if lines[u] & set(in_k) or not lines[u] & set(in_v):
            continue
        touched = torch.zeros((H, hs), dtype=torch.bool, device="cuda")
        touched[:, 5] = True
        touched[[h for h in range(H) if h * kv // H == kv - 1], hs - 1] = True
        got = out[u].float()
        assert torch.equal(out[u][~touched].view(torch.uint8), clean[u][~touched].view(torch.uint8))
        assert bool(got[touched].isnan().all()) if math.isnan(value) else bool((got[touched] == value).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pairs_heads", [(4, 4), (32, 2)])
def test_scores_of_minus_infinity_in_a_tree(dtype, pairs_heads):
    """A token all of whose scores but one are -inf, and tokens beside it."""
    H, kv = pairs_heads
    pool, rows, _, _ = build(dtype, H, kv, 64, 16, [(0, [12])], seed=1)
    trees = [[-1, 0, 1, 0, 3, 3, 2, 5]]
    index, starts, parents, B = call_of([0], trees)
    q = torch.ones((B, H, 64), device="cuda").to(DT[dtype])
    page = int(pool.table[0, 0])
    pool.k[0, page, :, :11, 0] = -float("inf")     # every key but token 7's
    out = pool.tree_attention(q, 0, index, starts, parents=parents)
    pool.check()
    want = pool.v[0, page, :, 11].repeat_interleave(H // kv, dim=0)
    half = torch.finfo(DT[dtype]).eps / 2
    assert bool(((out[7].double() - want.double()).abs() <= 2 * half * want.double().abs()).all())
    assert bool(out[:7].isnan().all())             # 0 / 0, as in the formula


def test_tree_attention_of_a_bad_page_reports_and_reads_nothing():
    pool, rows, _, _ = build("bf16", 4, 2, 64, 16, [(0, [50]), (0, [40])], seed=2)
    trees = trees_of("wide", [8, 8], 1)
    index, starts, parents, B = call_of([0, 1], trees)
    q = torch.randn((B, 4, 64), device="cuda").to(torch.bfloat16)
    lse = torch.empty((B, 4), device="cuda")
    pool.table[1, 0] = 10 ** 6
    out = pool.tree_attention(q, 0, index, starts, parents=parents, lse=lse)
    with pytest.raises(pkg.L2Error, match="outside the pool"):
        pool.check()
    check_attention(out[:8], lse[:8], q[:8], rows_seen(rows, [0], trees[:1]), "bf16", 1 / 8)
    k, v = (t.copy() for t in rows[1])
    k[:16] = v[:16] = 0
    check_attention(out[8:], lse[8:], q[8:], rows_seen([None, (k, v)], [1], trees[1:]), "bf16", 1 / 8)


@pytest.mark.parametrize("wrong", [
    dict(seqs=[0, 9]), dict(seqs=[-1, 1]), dict(starts=[1, 8, 16]), dict(starts=[0, 9, 8]), dict(starts=[0, 8, 17]),
    dict(starts=[0, -1, 16]), dict(parents={3: 3}), dict(parents={0: 0}), dict(parents={9: -2}), dict(parents={15: 8}), dict(lens=[7, 40])])
@pytest.mark.parametrize("many", [False, True])
def test_bad_index_arrays_are_reported_and_nothing_is_written(wrong, many):
    """many: as a call of so many sequences that a kernel plans it."""
    pad = 150 if many else 0
    pool, rows, _, _ = build("fp32", 4, 2, 16, 16, [(0, [50]), (0, [40])] + [(0, [3])] * pad, seed=2)
    trees = trees_of("wide", [8, 8], 1)
    seqs, starts = [0, 1], [0, 8, 16]
    parents = [p for t in trees for p in t]
    for r, p in wrong.get("parents", {}).items():
        parents[r] = p
    seqs = wrong.get("seqs", seqs) + list(range(2, 2 + pad))
    starts = wrong.get("starts", starts) + [16] * pad
    for s, n in enumerate(wrong.get("lens", [])):
        pool.lens[s] = n
    q = torch.randn((16, 4, 16), device="cuda")
    out = torch.full((16, 4, 16), 3.0, device="cuda")
    pool.tree_attention(q, 0, dev(seqs), dev(starts), parents=dev(parents), out=out)
    with pytest.raises(pkg.L2Error, match="bad index arrays"):
        pool.check()
    assert bool((out == 3.0).all())


def test_trees_larger_than_a_word_are_reported():
    pool, rows, _, _ = build("fp32", 2, 2, 16, 16, [(0, [100])], seed=2)
    q = torch.randn((65, 2, 16), device="cuda")
    out = torch.full_like(q, 3.0)
    pool.tree_attention(q, 0, dev([0]), dev([0, 65]), out=out)
    with pytest.raises(pkg.L2Error, match="bad index arrays"):
        pool.check()
    assert bool((out == 3.0).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_captured_tree_step_follows_lengths_trees_and_rows(dtype):
    """One graph, replayed for other sequences, trees and numbers of rows, with another call of the same pool between."""
    H, kv, hs = 8, 2, 64
    pool, rows, _, _ = build(dtype, H, kv, hs, 16, [(0, [n]) for n in (100, 30, 64, 5000)], seed=6)
    room = 48
    index, starts, parents = dev([0, 0]), dev([0, 0, 0]), dev([0] * room)
    q = torch.randn((room, H, hs), device="cuda").to(DT[dtype])
    out = torch.zeros((room, H, hs), device="cuda").to(DT[dtype])
    lse = torch.zeros((room, H), device="cuda")
    pool.tree_attention(q, 0, index, starts, parents=parents, out=out, lse=lse)   # warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.tree_attention(q, 0, index, starts, parents=parents, out=out, lse=lse)
    for turn, (order, sizes) in enumerate([([0, 1], [20, 28]), ([3, 2], [40, 1]), ([2, 0], [0, 7]), ([1, 3], [30, 18])]):
        trees = trees_of("wide", sizes, turn)
        i, s, p, B = call_of(order, trees)
        index.copy_(i)
        starts.copy_(s)
        parents[:B].copy_(p)
        q.normal_()
        out.fill_(2.0)
        graph.replay()
        pool.attention(q[:4], 0)   # another call's workspace
        pool.check()
        check_attention(out[:B], lse[:B], q[:B], rows_seen(rows, order, trees), dtype, 1 / 8)
        assert bool((out[B:] == 2.0).all())


def test_two_streams_and_dropped_arguments():
    pool, rows, _, _ = build("bf16", 8, 2, 64, 16, [(0, [n]) for n in (900, 300)], seed=8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    trees = trees_of("deep", [30, 20], 4)
    index, starts, parents, B = call_of([0, 1], trees)
    q = torch.randn((B, 8, 64), device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    outs = []
    for turn in range(6):
        st = streams[turn % 2]
        with torch.cuda.stream(st):
            mine = [t.clone() for t in (q, index, starts, parents)]
        outs.append(pool.tree_attention(mine[0], 0, mine[1], mine[2], parents=mine[3], stream=st))
        del mine
        torch.empty(B * 8 * 64, device="cuda").fill_(float("nan"))   # memory that came free is written to
    torch.cuda.synchronize()
    pool.check()
    want = pool.tree_attention(q, 0, index, starts, parents=parents)
    for out in outs:
        assert torch.equal(out.view(torch.uint8), want.view(torch.uint8))


# -- acceptance ----------------------------------------------------------------

def filled(dtype, L, n_pages, kv, ps, hs, lens, max_pages, order="head"):
    """A pool whose sequences hold `lens` rows, appended in turns so that their pages mix, and its plain statement."""
    pool = make_pool(DT[dtype], L, n_pages, kv, ps, hs, len(lens), max_pages, order)
    ref = pages_ref.RefPool(n_pages, ps, len(lens), max_pages)
    have = [0] * len(lens)
    while have != list(lens):
        seqs = [s for s in range(len(lens)) if have[s] < lens[s]]
        counts = [min(lens[s] - have[s], 1 + (3 * s + have[s]) % 5) for s in seqs]
        assert ref.append(seqs, counts) is not None
        rows = torch.randn((L, sum(counts), kv, hs), device="cuda").to(DT[dtype])
        pool.append(rows, -rows, dev(seqs), dev(np.concatenate([[0], np.cumsum(counts)])))
        for s, c in zip(seqs, counts):
            have[s] += c
    pool.check()
    return pool, ref


def positions(pool, s, n):
    t = pool.table[s].cpu().numpy()
    return (torch.tensor([int(t[i // pool.page_size]) for i in range(n)], device="cuda", dtype=torch.long),
            torch.tensor([i % pool.page_size for i in range(n)], device="cuda", dtype=torch.long))


def expect(pool, ref, order, sizes, paths):
    """What the pool's books and rows are after the paths were kept."""
    k, v = pool.k.clone(), pool.v.clone()
    for s, n, path in zip(order, sizes, paths):
        old = int(ref.lens[s])
        base = old - n
        page, at = positions(pool, s, old)
        for x in (k, v):
            held = x.permute(1, 3, 0, 2, 4)[page, at]          # a copy: [position][layer][head][value]
            src = [base + j for j in path]
            x.permute(1, 3, 0, 2, 4)[page[base:base + len(path)], at[base:base + len(path)]] = held[src]
        now = base + len(path)
        for c in range(-(-now // ref.ps), ref.held(s)):
            ref.refs[ref.table[s, c]] -= 1
        ref.lens[s] = now
    return k, v


def same(pool, ref, k, v):
    assert pool.lens.cpu().numpy().tolist() == ref.lens.tolist()
    assert pool.refs.cpu().numpy().tolist() == ref.refs.tolist()
    assert torch.equal(pool.k.view(torch.uint8), k.view(torch.uint8)) and torch.equal(pool.v.view(torch.uint8), v.view(torch.uint8))


ACCEPT = [
    # dtype, layers, kv, page size, head size, order in memory, (committed, drafted)
    ("fp32", 3, 4, 16, 8, "head", [(100, 7)]),
    ("bf16", 2, 3, 7, 48, "row", [(33, 16), (0, 64), (12, 1), (5, 0), (20, 40)]),
    ("fp16", 5, 2, 1, 64, "head", [(3, 20), (9, 5), (0, 3)]),
    ("fp32", 1, 1, 32, 128, "row", [(31, 64), (32, 64), (33, 64)]),
    ("bf16", 2, 2, 128, 8, "head", [(100, 50)] * 9),
]


@pytest.mark.parametrize("likely", [0.0, 0.6, 1.0])
@pytest.mark.parametrize("case", range(len(ACCEPT)))
def test_accepted_paths_and_what_is_left(case, likely):
    """likely: how often a token is what its parent's target says."""
    dtype, L, kv, ps, hs, order_in, seqs = ACCEPT[case]
    rng = np.random.default_rng(case * 10 + int(10 * likely))
    pool, ref = filled(dtype, L, 400, kv, ps, hs, [a + b for a, b in seqs], max(400 // ps, 140 // ps + 1), order_in)
    order = [int(s) for s in rng.permutation(len(seqs))]
    sizes = [seqs[s][1] for s in order]
    trees = [tree_ref.random_tree(rng, n, back=4) for n in sizes]
    tokens, targets, paths, follow = [], [], [], []
    for parents in trees:
        tar = [int(x) for x in rng.integers(0, 50, len(parents))]
        tok = [tar[p] if p >= 0 and rng.random() < likely else int(rng.integers(0, 50)) for p in parents]
        path, nxt = tree_ref.accepted(parents, tok, tar)
        tokens += tok
        targets += tar
        paths.append(path)
        follow.append(nxt)
    index, starts, parents, B = call_of(order, trees)
    k, v = expect(pool, ref, order, sizes, paths)
    # five more rows, behind the last tree: nobody's
    path, counts, nxt = pool.accept(dev(tokens + [1] * 5), dev(targets + [1] * 5), index, starts, parents=torch.cat([parents, dev([0] * 5)]))
    pool.check()
    assert counts.tolist() == [len(p) for p in paths] and nxt.tolist() == follow
    assert path.tolist() == [x for p, n in zip(paths, sizes) for x in p + [-1] * (n - len(p))] + [-1] * 5
    same(pool, ref, k, v)
    # the sequences go on
    rows = torch.randn((L, len(order), kv, hs), device="cuda").to(DT[dtype])
    assert ref.append(order, [1] * len(order)) is not None
    pool.append(rows, rows, index)
    pool.check()
    assert pool.lens.cpu().numpy().tolist() == ref.lens.tolist() and pool.refs.cpu().numpy().tolist() == ref.refs.tolist()


@pytest.mark.parametrize("case", range(len(ACCEPT)))
def test_given_paths_are_kept(case):
    dtype, L, kv, ps, hs, order_in, seqs = ACCEPT[case]
    rng = np.random.default_rng(case)
    pool, ref = filled(dtype, L, 400, kv, ps, hs, [a + b for a, b in seqs], max(400 // ps, 140 // ps + 1), order_in)
    order = [int(s) for s in rng.permutation(len(seqs))]
    sizes = [seqs[s][1] for s in order]
    # none, all, the last one, any
    paths = []
    for i, n in enumerate(sizes):
        some = sorted(rng.choice(n, rng.integers(0, n + 1), replace=False).tolist()) if n else []
        paths.append([[], list(range(n)), [n - 1] if n else [], some][(i + case) % 4] if len(seqs) > 1 else some)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    given = [x for p, n in zip(paths, sizes) for x in p + [77] * (n - len(p))]   # entries behind a path are not looked at
    k, v = expect(pool, ref, order, sizes, paths)
    pool.keep(dev(given + [5, 5]), dev([len(p) for p in paths]), dev(order), dev(starts))
    pool.check()
    same(pool, ref, k, v)


def test_rows_move_over_one_another():
    """Paths whose rows go where other accepted rows come from, longer than one batch of the copy."""
    pool, ref = filled("fp32", 2, 60, 2, 4, 16, [70, 40], 20)
    paths = [[0] + list(range(2, 40, 2)) + list(range(41, 64)), list(range(1, 30))]
    sizes = [64, 30]
    k, v = expect(pool, ref, [0, 1], sizes, paths)
    given = [x for p, n in zip(paths, sizes) for x in p + [0] * (n - len(p))]
    pool.keep(dev(given), dev([len(p) for p in paths]), dev([0, 1]), dev([0, 64, 94]))
    pool.check()
    same(pool, ref, k, v)


def test_acceptance_that_cannot_be_done_changes_nothing_and_accepts_nothing():
    pool, ref = filled("fp32", 2, 30, 2, 4, 8, [20, 13, 6], 8)
    parents = [-1, 0, 0, 1, -1, 0, 1]
    tokens, targets = [5, 6, 7, 8, 5, 6, 7], [7, 1, 1, 1, 6, 7, 9]   # paths [0, 2] and [0, 1, 2]

    def refused(text, seqs=(0, 1), starts=(0, 4, 7), parents=parents, prepare=None, undo=None):
        if prepare:
            prepare()
        before = [t.clone() for t in (pool.k, pool.v, pool.refs, pool.lens, pool.table)]
        out = torch.full((7 + 4,), 9, dtype=torch.int32, device="cuda")
        made = pool._made
        pool._made = lambda n, stream: out
        try:
            pool.accept(dev(tokens), dev(targets), dev(seqs), dev(starts), parents=dev(parents))
        finally:
            pool._made = made
        with pytest.raises(pkg.L2Error, match=text):
            pool.check()
        for a, b in zip(before, (pool.k, pool.v, pool.refs, pool.lens, pool.table)):
            assert torch.equal(a, b)
        n = len(seqs)
        assert bool((out[:7] == -1).all()) and bool((out[7:7 + n] == 0).all()) and bool((out[7 + n:] == -1).all())   # nothing is accepted
        if undo:
            undo()

    for bad in (dict(seqs=(0, 0)), dict(seqs=(0, 3)), dict(seqs=(-1, 1)), dict(starts=(1, 4, 7)), dict(starts=(0, 4, 8)), dict(starts=(0, 5, 4)),
                dict(parents=[-1, 0, 2, 1, -1, 0, 1]), dict(parents=[-1, 0, 0, 1, 0, 0, 1]), dict(parents=[-1, 0, 0, 1, -1, -2, 1])):
        refused("bad index arrays", **bad)
    # more rows than the sequence holds
    refused("bad index arrays", prepare=lambda: pool.lens[1:2].fill_(2), undo=lambda: pool.lens[1:2].fill_(13))
    # a page that rows move into is another sequence's too; a page outside the pool; a page nobody holds
    page = int(pool.table[0, 4])
    refused("inconsistent", prepare=lambda: pool.refs[page:page + 1].fill_(2), undo=lambda: pool.refs[page:page + 1].fill_(1))
    refused("inconsistent", prepare=lambda: pool.refs[page:page + 1].fill_(0), undo=lambda: pool.refs[page:page + 1].fill_(1))
    refused("outside the pool", prepare=lambda: pool.table[0, 4:5].fill_(-5), undo=lambda: pool.table[0, 4:5].fill_(page))
    # given paths: not ascending, past the tree, too many
    for path, counts in (([0, 0, 1, 1, 0, 0, 0], [2, 1]), ([1, 0, 2, 3, 0, 0, 0], [2, 1]), ([0, 4, 2, 3, 0, 0, 0], [2, 1]), ([0, 1, 2, 3, 0, 1, 3], [1, 3]),
                         ([-1, 0, 2, 3, 0, 0, 0], [2, 1]), ([0, 1, 2, 3, 0, 1, 2], [5, 1]), ([0, 1, 2, 3, 0, 1, 2], [1, -1])):
        before = [t.clone() for t in (pool.k, pool.v, pool.refs, pool.lens, pool.table)]
        pool.keep(dev(path), dev(counts), dev([0, 1]), dev([0, 4, 7]))
        with pytest.raises(pkg.L2Error, match="bad index arrays"):
            pool.check()
        for a, b in zip(before, (pool.k, pool.v, pool.refs, pool.lens, pool.table)):
            assert torch.equal(a, b)
    # and the call itself still works
    k, v = expect(pool, ref, [0, 1], [4, 3], [[0, 2], [0, 1, 2]])
    path, counts, nxt = pool.accept(dev(tokens), dev(targets), dev([0, 1]), dev([0, 4, 7]), parents=dev(parents))
    pool.check()
    assert path.tolist() == [0, 2, -1, -1, 0, 1, 2] and counts.tolist() == [2, 3] and nxt.tolist() == [1, 9]
    same(pool, ref, k, v)


def test_pages_shared_after_the_draft_are_given_back_by_one_holder():
    """A fork of a sequence with its drafted rows: whole pages of them are shared, so rows may not move into those, but
    they may be dropped down to a page's end."""
    pool, ref = filled("fp32", 1, 30, 1, 4, 8, [16, 0], 8)
    pool.fork(dev([0]), dev([1]))
    pool.check()
    before = pool.k.clone()
    pool.keep(dev([1] + [0] * 5), dev([1]), dev([0]), dev([0, 6]))       # into a shared page
    with pytest.raises(pkg.L2Error, match="inconsistent"):
        pool.check()
    pool.keep(dev([0] * 6), dev([1]), dev([0]), dev([0, 6]))             # leaves a shared page partly filled
    with pytest.raises(pkg.L2Error, match="inconsistent"):
        pool.check()
    pool.keep(dev([0, 1] + [0] * 4), dev([2]), dev([0]), dev([0, 6]))    # 12 rows: three whole pages
    pool.check()
    assert pool.lens.tolist() == [12, 16] and torch.equal(pool.k, before)
    refs = pool.refs.cpu().numpy()
    t = pool.table.cpu().numpy()
    assert [int(refs[p]) for p in t[1, :4]] == [2, 2, 2, 1]


def test_acceptance_in_a_graph_and_on_a_stream():
    pool, ref = filled("bf16", 3, 200, 2, 16, 64, [100] * 4, 12)
    parents = [-1, 0, 0, 1, 1, 2, 2, 3]
    index, starts = dev(range(4)), dev(np.arange(5) * 8)
    tokens, targets = dev([0] * 32), dev([0] * 32)
    par = dev(parents * 4)
    st = torch.cuda.Stream()
    saved = [t.clone() for t in (pool.k, pool.v, pool.refs, pool.lens)]
    torch.cuda.synchronize()
    pool.accept(tokens, targets, index, starts, parents=par, stream=st)   # warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        path, counts, nxt = pool.accept(tokens, targets, index, starts, parents=par)
    rng = np.random.default_rng(0)
    for _ in range(4):
        for t, s in zip((pool.k, pool.v, pool.refs, pool.lens), saved):
            t.copy_(s)
        ref.lens[:] = saved[3].cpu().numpy()
        ref.refs[:] = saved[2].cpu().numpy()
        tok, tar = rng.integers(0, 3, 32), rng.integers(0, 3, 32)
        tokens.copy_(dev(tok))
        targets.copy_(dev(tar))
        want = [tree_ref.accepted(parents, tok[8 * i:8 * i + 8], tar[8 * i:8 * i + 8]) for i in range(4)]
        k, v = expect(pool, ref, range(4), [8] * 4, [w[0] for w in want])
        graph.replay()
        pool.check()
        assert counts.tolist() == [len(w[0]) for w in want] and nxt.tolist() == [w[1] for w in want]
        same(pool, ref, k, v)


def test_the_largest_acceptance():
    """1024 sequences in one call, trees of none to 40 tokens, some sharing committed pages."""
    rng = np.random.default_rng(3)
    n, ps = 1024, 8
    pool = make_pool(F32, 1, 9000, 1, ps, 4, n, 10)
    ref = pages_ref.RefPool(9000, ps, n, 10)
    pre = [int(x) for x in rng.integers(0, 30, n)]
    sizes = [int(x) for x in rng.integers(0, 41, n)]
    counts = [a + b for a, b in zip(pre, sizes)]
    assert ref.append(range(n), counts) is not None
    rows = torch.randn((1, sum(counts), 1, 4), device="cuda")
    pool.append(rows, rows, dev(range(n)), dev(np.concatenate([[0], np.cumsum(counts)])))
    trees = [tree_ref.random_tree(rng, m, back=3) for m in sizes]
    tar = [rng.integers(0, 4, m) for m in sizes]
    tok = [rng.integers(0, 4, m) for m in sizes]
    want = [tree_ref.accepted(*x) for x in zip(trees, tok, tar)]
    index, starts, parents, B = call_of(range(n), trees)
    k, v = expect(pool, ref, range(n), sizes, [w[0] for w in want])
    path, cnt, nxt = pool.accept(dev(np.concatenate(tok)), dev(np.concatenate(tar)), index, starts, parents=parents)
    pool.check()
    assert cnt.tolist() == [len(w[0]) for w in want] and nxt.tolist() == [w[1] for w in want]
    same(pool, ref, k, v)
