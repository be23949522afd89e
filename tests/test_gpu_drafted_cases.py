"""Calls on drafted tokens that the documentation allows at the edges: uneven heads with several warps to a tile, tables with room for very long
sequences, offsets past 32 bits, two graphs at once, the largest calls.  Tolerances are those of the operators' own tests."""
import math

import numpy as np
import pytest

from tests import tree_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402
from tests.test_gpu_pages import DT, build, check_attention, dev  # noqa: E402
from tests.test_gpu_rope import check as check_rope  # noqa: E402
from tests.test_gpu_tree import call_of, rows_seen, trees_of  # noqa: E402


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("H,kv,hs,ps,seqs", [
    (10, 4, 64, 16, [(200, 40), (33, 64), (0, 17)]),         # three query heads or two to a KV head, four warps
    (5, 2, 128, 24, [(500, 20), (70, 22), (1, 64)]),
    (7, 3, 32, 16, [(90, 9), (300, 10)]),                    # two warps
    (7, 3, 128, 16, [(90, 9), (300, 10)]),
    (9, 9, 64, 32, [(100, 33), (5, 30), (60, 1), (0, 64)]),  # two warps, trees that need one and four
    (16, 2, 128, 128, [(3000, 4), (2900, 5)]),
    (64, 8, 64, 64, [(1000, 3), (12, 8), (500, 6)]),
    (16, 1, 8, 16, [(3000, 64), (1, 1)]),                    # 1024 pairs of one KV head
])
def test_teams_of_warps_and_uneven_heads(H, kv, hs, ps, seqs, dtype):
    pool, rows, _, _ = build(dtype, H, kv, hs, ps, [(0, [p + n]) for p, n in seqs], seed=H + hs)
    order = list(np.random.default_rng(1).permutation(len(seqs)))
    for kind in ("wide", "chain"):
        trees = trees_of(kind, [seqs[s][1] for s in order], 3)
        index, starts, parents, B = call_of(order, trees)
        q = torch.randn((B, H, hs), device="cuda").to(DT[dtype]) * 2
        lse = torch.empty((B, H), device="cuda")
        out = pool.tree_attention(q, 0, index, starts, parents=parents, lse=lse)
        pool.check()
        check_attention(out, lse, q, rows_seen(rows, order, trees), dtype, 1 / math.sqrt(hs))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("hs,committed", [(40, [0, 30, 1, 700]), (128, [2500, 3, 64, 0])])
def test_an_odd_number_of_very_many_pairs(hs, committed, dtype):
    """255 rows of 33 heads: the last pair stands alone, and rows behind the last tree lie beside written ones."""
    H, kv, sizes = 33, 3, [63, 64, 62, 63]
    pool, rows, _, _ = build(dtype, H, kv, hs, 16, [(0, [p + n]) for p, n in zip(committed, sizes)], seed=hs)
    trees = trees_of("wide", sizes, hs)
    index, starts, parents, B = call_of(range(4), trees)
    room = 255
    parents = torch.cat([parents, torch.full((room - B,), -7, dtype=torch.int32, device="cuda")])
    g = torch.Generator(device="cuda").manual_seed(hs)
    q = torch.randn((room, H, hs), generator=g, device="cuda").to(DT[dtype])
    out = torch.full((room, H, hs), 7.0, device="cuda").to(DT[dtype])
    lse = torch.full((room, H), 7.0, device="cuda")
    pool.tree_attention(q, 0, index, starts, parents=parents, out=out, lse=lse)
    pool.check()
    check_attention(out[:B], lse[:B], q[:B], rows_seen(rows, range(4), trees), dtype, 1 / math.sqrt(hs))
    assert bool((out[B:] == 7.0).all()) and bool((lse[B:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_tables_with_room_for_very_long_sequences(dtype):
    """Sequences as long as their tables would be too many keys to number in 32 bits, so a kernel plans the call by its lengths."""
    pool, rows, _, _ = build(dtype, 16, 2, 64, 16, [(0, [n]) for n in (300, 70, 5)], seed=4)
    wide = torch.zeros((3, 1 << 20), dtype=torch.int32, device="cuda")
    wide[:, :pool.max_pages] = pool.table
    pool = pkg.PagePool.from_tensors(pool.k, pool.v, pool.refs, pool.lens, wide)
    trees = trees_of("deep", [64, 30, 5], 2)
    index, starts, parents, B = call_of([0, 1, 2], trees)
    q = torch.randn((B, 16, 64), device="cuda").to(DT[dtype])
    lse = torch.empty((B, 16), device="cuda")
    out = pool.tree_attention(q, 0, index, starts, parents=parents, lse=lse)
    pool.check()
    check_attention(out, lse, q, rows_seen(rows, [0, 1, 2], trees), dtype, 1 / 8)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_pages_past_32_bits(dtype):
    """Attention and acceptance over pages whose bytes lie more than 2^32 from the pool's first."""
    small, rows, _, _ = build(dtype, 8, 2, 64, 16, [(0, [90]), (0, [40])], seed=9)
    apart = (1 << 30) // small.k.element_size()                     # elements from page to page
    flat = [torch.zeros(apart * small.n_pages, dtype=DT[dtype], device="cuda") for _ in range(2)]
    st = (apart * small.n_pages, apart, 16 * 64, 64, 1)
    k, v = (t.as_strided(small.k.shape, st) for t in flat)
    k.copy_(small.k)
    v.copy_(small.v)
    refs = torch.zeros_like(small.refs)
    for s, n in ((0, 90), (1, 40)):
        refs[small.table[s, :-(-n // 16)].long()] = 1
    pool = pkg.PagePool.from_tensors(k, v, refs, small.lens, small.table)
    assert int(pool.table[0, :6].max()) * (1 << 30) > 1 << 32
    trees = trees_of("wide", [40, 20], 2)
    index, starts, parents, B = call_of([0, 1], trees)
    q = torch.randn((B, 8, 64), device="cuda").to(DT[dtype])
    lse = torch.empty((B, 8), device="cuda")
    out = pool.tree_attention(q, 0, index, starts, parents=parents, lse=lse)
    pool.check()
    check_attention(out, lse, q, rows_seen(rows, [0, 1], trees), dtype, 1 / 8)
    path = [0, 5, 9, 30, 39]
    pool.keep(dev(path + [0] * 35 + [19] + [0] * 19), dev([5, 1]), index, starts)
    pool.check()
    table = pool.table.cpu().numpy()
    for s, base, kept in ((0, 50, path), (1, 20, [19])):
        for j, u in enumerate(kept):
            at = base + j
            for pages, mine in zip((pool.k, pool.v), rows[s]):
                got = pages[0, int(table[s, at // 16]), :, at % 16]
                assert torch.equal(got.double().cpu(), torch.from_numpy(mine[base + u])), (s, j)
    assert pool.lens.tolist() == [55, 21]


def test_rows_histories_and_masks_past_32_bits():
    V, n = 64, 2
    far = (1 << 31) + 64                                            # elements from one to the next
    history = torch.zeros(far + 8, dtype=torch.int32, device="cuda").as_strided((n, 8), (far, 1))
    history[1] = dev([7, 7, 9, 0, 0, 0, 0, 0])
    rules = pkg.TokenRules(V, history, dev([0, 3]), frequency=torch.ones(n, device="cuda"))
    logits = torch.zeros(far + V, dtype=torch.bfloat16, device="cuda").as_strided((n, V), (far, 1))
    masks = torch.full((far + 2,), -1, dtype=torch.int32, device="cuda").as_strided((n, 2), (far, 1))
    masks[1, 1] = 1                                                 # of tokens 32..63 only 32
    out = torch.full((far + V,), 3.0, dtype=torch.bfloat16, device="cuda").as_strided((n, V), (far, 1))
    logits[1] = 2.0
    rules.apply(logits, masks=masks, out=out)
    rules.check()
    assert bool((out[0] == 0).all())
    want = [2.0] * 33 + [-math.inf] * 31
    want[7], want[9] = 0.0, 1.0
    assert out[1].tolist() == want
    del history, logits, masks, out, rules
    rope = pkg.Rope(64, layout="half")
    x = torch.zeros(3 * (1 << 30), dtype=torch.bfloat16, device="cuda").as_strided((3, 2, 64), (1 << 30, 64, 1))
    x.normal_()
    pos = dev([5, 70000, 123])
    y, _ = rope.apply(pos, x)
    check_rope(y, x, pos, rope)
    rope.apply(pos, x, out_q=x)
    assert torch.equal(x, y)


def test_two_graphs_of_trees_and_calls_between():
    pool, rows, _, _ = build("bf16", 16, 2, 64, 16, [(0, [n]) for n in (5000, 700, 64)], seed=8)
    graphs = []
    for kind, order, sizes in (("wide", [0, 1], [64, 30]), ("deep", [2, 0], [20, 7])):
        trees = trees_of(kind, sizes, 3)
        index, starts, parents, B = call_of(order, trees)
        q = torch.randn((B, 16, 64), device="cuda").to(torch.bfloat16)
        pool.tree_attention(q, 0, index, starts, parents=parents)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        lse = torch.zeros((B, 16), device="cuda")
        with torch.cuda.graph(g):
            out = pool.tree_attention(q, 0, index, starts, parents=parents, lse=lse)
        graphs.append((g, q, out, lse, rows_seen(rows, order, trees)))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for turn in range(4):
        for st, (g, *_) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        pool.attention(torch.randn((3, 16, 64), device="cuda").to(torch.bfloat16), 0)
    torch.cuda.synchronize()
    pool.check()
    for _, q, out, lse, seen in graphs:
        check_attention(out, lse, q, seen, "bf16", 1 / 8)


def test_the_largest_calls():
    """1024 rows and 1024 heads of one row; 65535 rows of rules; many rows of one token each in rotary positions."""
    pool, rows, _, _ = build("fp32", 1024, 16, 8, 16, [(0, [40])], seed=2)
    q = torch.randn((3, 1024, 8), device="cuda")
    lse = torch.empty((3, 1024), device="cuda")
    out = pool.tree_attention(q, 0, dev([0]), dev([0, 3]), lse=lse)
    pool.check()
    check_attention(out, lse, q, rows_seen(rows, [0], [tree_ref.chain(3)]), "fp32", 1 / math.sqrt(8))
    V, n = 70, 65535
    hist = torch.randint(0, V, (n, 5), dtype=torch.int32, device="cuda")
    rules = pkg.TokenRules(V, hist, torch.full((n,), 5, dtype=torch.int32, device="cuda"), presence=torch.ones(n, device="cuda"))
    x = torch.randn((n, V), device="cuda")
    got = rules.apply(x, seqs=torch.arange(n, dtype=torch.int32, device="cuda"), starts=torch.arange(n + 1, dtype=torch.int32, device="cuda"))
    rules.check()
    seen = torch.zeros((n, V), device="cuda").scatter_(1, hist.long(), 1.0)
    assert torch.equal(got, x - seen)
    rope = pkg.Rope(8)
    x = torch.randn((1 << 20, 1, 8), device="cuda").to(torch.float16)
    pos = torch.arange(1 << 20, dtype=torch.int32, device="cuda")
    y, _ = rope.apply(pos, x)
    check_rope(y, x, pos, rope)
