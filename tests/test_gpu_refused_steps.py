"""Steps with drafted tokens whose rows were refused, enqueued to their end without a wait: an append that a full pool cannot take is followed by its
other layers, attention and acceptance.  What the sequences had committed stays, bit for bit, whatever other sequences do in between."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402
from tests.test_gpu_pages import DT, dev  # noqa: E402

L, KV, HS = 2, 2, 16


def pool_of(lens, n_pages, ps, max_pages=16, dtype="fp32"):
    """Sequences of so many rows in every layer, taken in order, and two more that are empty."""
    pool = pkg.PagePool(L, n_pages, KV, ps, HS, len(lens) + 2, max_pages, dtype=DT[dtype])
    x = torch.randn((2, L, sum(lens), KV, HS), device="cuda").to(DT[dtype])
    pool.append(x[0], x[1], dev(range(len(lens))), dev(np.concatenate([[0], np.cumsum(lens)])))
    pool.check()
    return pool


def rows(n, pool):
    return torch.randn((2, L, n, KV, HS), device="cuda").to(pool.dtype)


def append(pool, x, seqs, starts, layers=range(L)):
    for layer in layers:
        pool.append(x[0, layer], x[1, layer], dev(seqs), dev(starts), layer=layer)


def held(pool, s):
    """A sequence's rows, [K or V][layer][row]."""
    n, t = int(pool.lens[s]), pool.table[s].tolist()
    page = torch.tensor([t[i // pool.page_size] for i in range(n)], device="cuda", dtype=torch.long)
    at = torch.tensor([i % pool.page_size for i in range(n)], device="cuda", dtype=torch.long)
    return torch.stack([x.permute(1, 3, 0, 2, 4)[page, at].transpose(0, 1) for x in (pool.k, pool.v)])


def books(pool):
    return [t.clone() for t in (pool.k, pool.v, pool.refs, pool.lens, pool.table)]


def same(before, pool):
    return all(torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(before, books(pool)))


def take(pool, how, seqs, starts, fits=100):
    """Chains whose first `fits` tokens the model agrees with are accepted, or all of their tokens but the second kept."""
    sizes = [b - a for a, b in zip(starts, starts[1:])]
    if how == "accept":
        tokens = [u for n in sizes for u in range(n)]
        targets = [u + 1 if u + 1 < fits else 0 for n in sizes for u in range(n)]
        return pool.accept(dev(tokens), dev(targets), dev(seqs), dev(starts))
    path = [x for n in sizes for x in [0] + list(range(2, n)) + [0] * (n > 1)]
    pool.keep(dev(path), dev([n - (n > 1) for n in sizes]), dev(seqs), dev(starts))


def nothing(got, rows, n):
    path, counts, following = got
    assert path.tolist() == [-1] * rows and counts.tolist() == [0] * n and following.tolist() == [-1] * n


def cleared(pool, match):
    with pytest.raises(pkg.L2Error, match=match):
        pool.check()


@pytest.mark.parametrize("how", ["accept", "keep"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,ps", [((100, 37), 16), ((96, 64), 32), ((7, 9), 1), ((60, 20), 64)])
def test_a_step_that_does_not_fit_leaves_what_was_committed(lens, ps, dtype, how):
    pool = pool_of(lens, sum(-(-n // ps) for n in lens), ps, max_pages=-(-max(lens) // ps) - (-60 // ps) + 1, dtype=dtype)   # no page is free
    before = books(pool)
    seqs, starts = [1, 0], [0, 7, 14]
    if any(n % ps and n % ps + 7 <= ps for n in lens):     # rows left in the last page: trees that go past it
        starts = [0, 7, 7 + 60]
    n = starts[-1]
    x = rows(n, pool)
    append(pool, x, seqs, starts)
    q = torch.randn((n, 4, HS), device="cuda").to(pool.dtype)
    pool.tree_attention(q, 0, dev(seqs), dev(starts))
    got = take(pool, how, seqs, starts, fits=3)
    cleared(pool, "free pages")
    assert same(before, pool)
    if how == "accept":
        nothing(got, n, 2)
    # the status is clear, and still nothing was appended
    got = take(pool, how, seqs, starts)
    cleared(pool, "bookkeeping")
    assert same(before, pool)


@pytest.mark.parametrize("how", ["accept", "keep"])
def test_a_tree_that_is_accepted_whole_is_not_taken_from_committed_rows(how):
    pool = pool_of((40,), 5, 8)
    before = books(pool)
    append(pool, rows(4, pool), [0], [0, 4])
    if how == "accept":
        got = pool.accept(dev([0, 1, 2, 3]), dev([1, 2, 3, 4]), dev([0]), dev([0, 4]))
        nothing(got, 4, 1)
    else:
        pool.keep(dev(range(4)), dev([4]), dev([0]), dev([0, 4]))
    cleared(pool, "free pages")
    assert same(before, pool)


@pytest.mark.parametrize("how", ["accept", "keep"])
def test_another_sequences_step_in_between(how):
    """Two batches take turns on one pool: what was refused to the first stays refused after the second's success, which is none of its business."""
    pool = pool_of((30, 21), 8, 8)                        # one page is free
    old = held(pool, 0)
    append(pool, rows(12, pool), [0], [0, 12], layers=[0])    # needs two
    x = rows(5, pool)
    append(pool, x, [1], [0, 5])                          # fits
    k, v = pool.k.clone(), pool.v.clone()
    append(pool, rows(12, pool), [0], [0, 12], layers=[1])    # the refused step goes on
    assert torch.equal(pool.k, k) and torch.equal(pool.v, v)
    pool.status.zero_()
    before = books(pool)
    got = take(pool, how, [0], [0, 12])
    cleared(pool, "bookkeeping")
    assert same(before, pool)
    if how == "accept":
        nothing(got, 12, 1)
    mine = held(pool, 1)
    take(pool, how, [1], [0, 5])
    pool.check()
    assert torch.equal(held(pool, 0), old)
    assert torch.equal(held(pool, 1), mine if how == "accept" else mine[:, :, [i for i in range(26) if i != 22]])
    # both in one call: all of it or nothing
    append(pool, rows(40, pool), [0], [0, 40])
    pool.status.zero_()
    before = books(pool)
    take(pool, how, [1, 0], [0, 2, 9])
    cleared(pool, "bookkeeping")
    assert same(before, pool)
    # an extension that succeeds is one's own again
    pool.free(dev([1]))
    x = rows(6, pool)
    append(pool, x, [0], [0, 6])
    pool.check()
    assert torch.equal(held(pool, 0), torch.cat([old, x], dim=2))
    take(pool, how, [0], [0, 6])
    pool.check()
    assert torch.equal(held(pool, 0), torch.cat([old, x if how == "accept" else x[:, :, [0, 2, 3, 4, 5]]], dim=2))


def test_a_step_before_the_refused_one_is_accepted():
    pool = pool_of((30, 21), 8, 8)
    old, x = held(pool, 1), rows(4, pool)
    append(pool, x, [1], [0, 4])                          # 25 rows: the last free page
    append(pool, rows(12, pool), [0], [0, 12])
    cleared(pool, "free pages")
    path, counts, following = take(pool, "accept", [1], [0, 4])
    pool.check()
    assert path.tolist() == [0, 1, 2, 3] and counts.tolist() == [4] and following.tolist() == [4]
    assert torch.equal(held(pool, 1), torch.cat([old, x], dim=2))


def test_rows_that_a_refusal_left_out_are_not_accepted():
    """A refused extension holds for the layers of every step under way: the sequences whose rows were left out are not whole."""
    pool = pool_of((30, 21), 10, 8)
    append(pool, rows(4, pool), [1], [0, 4], layers=[0])
    append(pool, rows(20, pool), [0], [0, 20])
    append(pool, rows(4, pool), [1], [0, 4], layers=[1])      # left out
    x = rows(3, pool)
    append(pool, x, [2], [0, 3])                              # a success of another sequence
    cleared(pool, "free pages")
    before = books(pool)
    nothing(take(pool, "accept", [1], [0, 4]), 4, 1)
    cleared(pool, "bookkeeping")
    assert same(before, pool)
    take(pool, "accept", [2], [0, 3])
    pool.check()
    # with the next rows those come out by a path that leaves them
    y = rows(2, pool)
    append(pool, y, [1], [0, 2])
    old = held(pool, 1)
    pool.keep(dev([4, 5, 0, 0, 0, 0]), dev([2]), dev([1]), dev([0, 6]))
    pool.check()
    assert torch.equal(held(pool, 1), torch.cat([old[:, :, :21], y], dim=2))


@pytest.mark.parametrize("whole", [False, True])
def test_rows_that_were_left_out_may_be_written_again(whole):
    """Once there is room: from the lowest layer on that they were left out of, or all layers at once."""
    pool = pkg.PagePool(4, 12, KV, 8, HS, 4, 16)
    x = torch.randn((2, 4, 51, KV, HS), device="cuda")
    pool.append(x[0], x[1], dev([0, 1]), dev([0, 30, 51]))    # 4 and 3 pages, five are free
    old = held(pool, 1)
    y, z = torch.randn((2, 4, 4, KV, HS), device="cuda"), torch.randn((2, 4, 40, KV, HS), device="cuda")
    append(pool, y, [1], [0, 4], layers=[0, 1])
    append(pool, z, [0], [0, 40], layers=[0])                 # five pages, four are free
    append(pool, y, [1], [0, 4], layers=[2])                  # left out
    append(pool, z[:, :, :9], [0], [0, 9], layers=[0, 1, 2, 3])
    append(pool, y, [1], [0, 4], layers=[3])                  # written, but the one below is not there
    cleared(pool, "free pages")
    before = books(pool)
    nothing(take(pool, "accept", [1], [0, 4]), 4, 1)
    cleared(pool, "bookkeeping")
    assert same(before, pool)
    if whole:
        pool.append(y[0], y[1], dev([1]), dev([0, 4]), extend=False)
    else:
        for layer in (2, 3):
            pool.append(y[0, layer], y[1, layer], dev([1]), dev([0, 4]), layer=layer)
    path, counts, following = take(pool, "accept", [1], [0, 4], fits=3)
    pool.check()
    assert counts.tolist() == [3] and torch.equal(held(pool, 1), torch.cat([old, y[:, :, :3]], dim=2))
    path, counts, following = take(pool, "accept", [0], [0, 9], fits=5)
    pool.check()
    assert counts.tolist() == [5]


def test_rows_of_a_refused_sequence_are_reported_once_others_succeed():
    pool = pool_of((30, 21), 8, 8)
    append(pool, rows(12, pool), [0], [0, 12], layers=[0])    # refused
    append(pool, rows(5, pool), [1], [0, 5])
    cleared(pool, "free pages")
    before = books(pool)
    append(pool, rows(12, pool), [0], [0, 12], layers=[1])
    cleared(pool, "bookkeeping")
    assert same(before, pool)


def test_a_refusal_goes_with_its_pages():
    """Compaction moves them, a fork copies a partly filled one, and one that was given back and taken again is a new sequence's."""
    pool = pool_of((9, 30, 21), 10, 8)
    append(pool, rows(20, pool), [1], [0, 20])               # refused
    pool.status.zero_()
    pool.free(dev([0]), compact=True)                        # sequence 1's last page (5) stays below 7 held; 2's move
    pool.fork(dev([1]), dev([0]))                            # its last page has 6 rows: copied
    pool.check()
    append(pool, rows(1, pool), [2], [0, 1])
    pool.check()
    for s in (0, 1):
        before = books(pool)
        nothing(take(pool, "accept", [s], [0, 7]), 7, 1)
        cleared(pool, "bookkeeping")
        assert same(before, pool)
    pool.free(dev([0, 1, 2]))
    x = rows(70, pool)
    append(pool, x, [3], [0, 70])                            # the pages that were held, too
    take(pool, "keep", [3], [0, 60])
    pool.check()
    assert torch.equal(held(pool, 3), x[:, :, [i for i in range(70) if i != 11]])
    pool.keep(dev(range(60)), dev([35]), dev([3]), dev([0, 60]))   # down to the page that sequence 1 ended in
    assert int(pool.table[3, 5]) == 5
    take(pool, "keep", [3], [0, 5])                          # and once more
    pool.check()
    assert int(pool.lens[3]) == 43


def test_a_refusal_that_moves_below_the_held_pages():
    pool = pool_of((33, 30, 21), 12, 8)
    append(pool, rows(20, pool), [2], [0, 20])               # refused: no page is free
    pool.status.zero_()
    old = held(pool, 2)
    pool.free(dev([0]), compact=True)
    pool.check()
    assert max(pool.table[2, :3].tolist()) < 7 and torch.equal(held(pool, 2), old)
    append(pool, rows(1, pool), [1], [0, 1])
    before = books(pool)
    nothing(take(pool, "accept", [2], [0, 7]), 7, 1)
    cleared(pool, "bookkeeping")
    assert same(before, pool)


def test_forks_that_share_their_last_page():
    """Both end with a whole page that they share; the one that got its rows goes on, the other was refused."""
    pool = pool_of((16,), 5, 8, max_pages=6)
    pool.fork(dev([0]), dev([1]))
    append(pool, rows(30, pool), [1], [0, 30])               # refused: three are free
    x = rows(9, pool)
    append(pool, x, [0], [0, 9])
    pool.status.zero_()
    before = books(pool)
    nothing(take(pool, "accept", [1], [0, 8]), 8, 1)
    cleared(pool, "bookkeeping")
    assert same(before, pool)
    old = held(pool, 1)
    take(pool, "keep", [0], [0, 9])
    pool.check()
    assert torch.equal(held(pool, 0), torch.cat([old, x[:, :, [0] + list(range(2, 9))]], dim=2)) and torch.equal(held(pool, 1), old)


def test_bad_calls_that_extend_refuse_their_sequences_too():
    pool = pool_of((12, 20), 20, 8, max_pages=4)
    append(pool, rows(14, pool), [0, 1], [0, 1, 14])         # sequence 1 would be longer than its table
    cleared(pool, "index")
    before = books(pool)
    for s in (0, 1):
        nothing(take(pool, "accept", [s], [0, 3]), 3, 1)
        cleared(pool, "bookkeeping")
        assert same(before, pool)
    append(pool, rows(2, pool), [0, 1], [0, 2, 2])           # sequence 0 alone gets rows
    take(pool, "accept", [0], [0, 2])
    pool.check()
    nothing(take(pool, "accept", [1], [0, 3]), 3, 1)
    cleared(pool, "bookkeeping")


def test_a_captured_step_that_is_refused_and_then_fits():
    pool = pool_of((30, 21), 8, 8)                           # 30 rows in 4 pages, 21 in 3; one is free
    old = held(pool, 0)
    x, seqs, starts = rows(12, pool), dev([0]), dev([0, 12])
    tokens, targets = dev(range(12)), dev([1, 2, 3] + [0] * 9)
    pool.accept(dev([0]), dev([0]), dev([2]), dev([0, 0]))   # loads the kernels
    pool.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for layer in range(L):
            pool.append(x[0, layer], x[1, layer], seqs, starts, layer=layer)
        path, counts, following = pool.accept(tokens, targets, seqs, starts)
    for _ in range(2):
        graph.replay()
        cleared(pool, "free pages")
        assert torch.equal(held(pool, 0), old)
        nothing((path, counts, following), 12, 1)
    pool.free(dev([1]))
    graph.replay()
    pool.check()
    assert counts.tolist() == [4] and following.tolist() == [0] and path.tolist() == [0, 1, 2, 3] + [-1] * 8
    assert torch.equal(held(pool, 0), torch.cat([old, x[:, :, :4]], dim=2))
