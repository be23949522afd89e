"""The paged cache on the GPU, call by call: what the documentation allows and other tests do not make.  Helpers and
tolerances are those of tests/test_gpu_pages.py."""
import math

import numpy as np
import pytest

from tests import pages_plan

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402,F401
from tests.test_gpu_pages import DT, check_wide, dev, wide_pool  # noqa: E402


def grouped(dtype, groups, lens, kv, hs, ps, seed, order="head"):
    """A pool whose sequences come in groups of (prefix, members) that share their prefix: whole pages by reference, the rest
    copied.  Returns the pool, the rows of a sequence in 64 bits, and the call's group arguments."""
    sizes, prefixes = [m for _, m in groups], [p for p, _ in groups]
    starts = np.concatenate([[0], np.cumsum(sizes)])
    firsts, prefix = np.repeat(starts[:-1], sizes), np.repeat(prefixes, sizes)
    pool, rows = wide_pool(dtype, len(firsts), kv, hs, ps, lens, [(int(f), int(p) // ps * ps) for f, p in zip(firsts, prefix)], seed=seed, order=order)
    for g, (p, m) in enumerate(groups):
        tail, a, b = p % ps, int(starts[g]), int(starts[g + 1])
        if tail and m > 1:
            pages = pool.table[a:b, p // ps].long()
            for t in (pool.k, pool.v):
                t[0, pages[1:], :, :tail] = t[0, pages[:1], :, :tail].expand(m - 1, -1, -1, -1)
    return pool, rows, dict(group_starts=dev(starts), prefix_lens=dev(prefixes))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(pages_plan.CROSSED)))
def test_blocks_that_go_on_to_another_item(case, dtype):
    """Blocks of the tensor-core role whose items leave the slots' tiles changed over (tests/test_attn_slots.py)."""
    groups, _, H, kv, hs = pages_plan.CROSSED[case]
    lens = pages_plan.crossed_lens(case)
    pool, rows, args = grouped(dtype, groups, lens, kv, hs, 64, seed=case)
    q = torch.randn((len(lens), H, hs), device="cuda").to(DT[dtype])
    lse = torch.empty((len(lens), H), device="cuda")
    out = pool.attention(q, 0, lse=lse, **args)
    pool.check()
    some = np.concatenate([[0], np.cumsum([m for _, m in groups])[:-1], [len(lens) - 1]])[:: max(1, len(groups) // 4)]
    check_wide(out, lse, q, rows, dtype, 1 / math.sqrt(hs), sorted({int(b) for b in some}))
    for _ in range(5):
        assert torch.equal(pool.attention(q, 0, **args), out)
    pool.check()


# heads, KV heads, head size, members, prefix, whether the tensor-core role takes the prefix
WEIGHTS = [(32, 4, 64, 40, 6400, True), (32, 32, 64, 40, 3456, True), (32, 32, 128, 40, 2048, True), (32, 4, 128, 40, 3200, True),
           (8, 2, 64, 3, 700, False), (8, 8, 128, 1, 1000, False)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(WEIGHTS)))
def test_weights_of_16_bit_caches_are_not_rounded_to_16_bits(case, dtype):
    """Whichever way a tile goes, a weight is two values of the type: off by at most w = 2^-16 (bf16: a half step of a half step)
    or 2^-22 (fp16), and in fp16 by 2^-38 of the largest.  Keys differ in one dimension, so a score is one exact product, off by
    the scaling alone, e = 8u of its size; a sum takes two products per 16 keys, each add at most 2u of the sum of w |v|.
    A single 16-bit value (half a step of the type on each weight) does not keep this where few keys matter."""
    H, kv, hs, members, prefix, tc = WEIGHTS[case]
    groups = [(prefix, members)]
    lens = prefix + np.arange(members) % 5
    assert bool(pages_plan.tc_blocks(groups, lens, H, kv, hs)) == tc
    pool, rows, args = grouped(dtype, groups, lens, kv, hs, 32, seed=case)
    pool.k[..., 1:] = 0
    q = torch.zeros((members, H, hs), device="cuda").to(DT[dtype])
    q[..., 0] = (torch.rand((members, H), device="cuda") * 2 + 3).to(DT[dtype])
    out = pool.attention(q, 0, scale=1.0, **args)
    pool.check()
    u, half, w2 = 2.0 ** -24, torch.finfo(DT[dtype]).eps / 2, 2.0 ** -16 if dtype == "bf16" else 2.0 ** -22
    heads = torch.arange(H, device="cuda") * kv // H
    worst = 0.0
    for b in range(0, members, 3):
        k, v = rows(b)
        n = len(k)
        x = k[:, heads, 0].T * q[b, :, 0].double()[:, None]
        w = torch.softmax(x, 1)
        want, mag = torch.einsum("ht,thd->hd", w, v[:, heads]), torch.einsum("ht,thd->hd", w, v[:, heads].abs())
        e = 8 * u * float(x.abs().max())
        rel = 2 * (e + 8 * u * float(x.abs().max())) + w2 + (n / 8 + 66) * 2 * u
        tiny = n * 2.0 ** -38 * float(v.abs().max()) + 2.0 ** -25 if dtype == "fp16" else 1e-38
        tol = rel * mag + half * (want.abs() + rel * mag) + tiny
        worst = max(worst, float(((out[b].double() - want).abs() / tol).max()))
    assert worst <= 1, worst


# -- a step's layers, with other calls between them ---------------------------

def small_pool(n_pages=6, layers=2):
    """Sequences 0 (6 rows) and 2 (7 rows) in pages of 4; 0 shares nothing."""
    pool = pkg.PagePool(layers, n_pages, 2, 4, 8, 6, 4)
    x = torch.randn((2, layers, 13, 2, 8), device="cuda")
    pool.append(x[0], x[1], dev([0, 2]), dev([0, 6, 13]))
    pool.check()
    return pool


def refused(pool, match):
    with pytest.raises(pkg.L2Error, match=match):
        pool.check()


@pytest.mark.parametrize("between", ["free", "fork", "free_compact"])
def test_a_refused_extension_holds_for_the_other_layers_whatever_succeeds_between(between):
    pool = small_pool()
    x = torch.randn((2, 9, 2, 8), device="cuda")
    pool.append(x[0], x[0], dev([0]), dev([0, 9]), layer=0)     # 15 rows: 2 more pages, both free
    pool.check()
    pool.append(x[1], x[1], dev([1]), dev([0, 9]), layer=0)     # no page is left
    refused(pool, "free pages")
    if between == "fork":
        pool.fork(dev([0]), dev([3]), dev([4]))                 # a whole page: no new one
    else:
        pool.free(dev([2]), compact=between == "free_compact")
    pool.check()
    k, v, lens = pool.k.clone(), pool.v.clone(), pool.lens.clone()
    pool.append(x[1], x[1], dev([1]), dev([0, 9]), layer=1)     # the refused step's other layer
    pool.append(x[1, :1], x[1, :1], dev([0]), layer=1, extend=False)
    torch.cuda.synchronize()
    assert torch.equal(pool.k, k) and torch.equal(pool.v, v) and torch.equal(pool.lens, lens)
    pool.status.zero_()
    # and one that succeeds ends it
    pool.free(dev([2]))
    pool.append(x[1, :3], x[1, :3], dev([1]), dev([0, 3]), layer=0)
    pool.append(x[0, :3], x[0, :3], dev([1]), dev([0, 3]), layer=1)
    pool.check()
    page = int(pool.table[1, 0])
    assert torch.equal(pool.k[0, page, :, :3], x[1, :3].transpose(0, 1)) and torch.equal(pool.k[1, page, :, :3], x[0, :3].transpose(0, 1))


def test_refused_calls_between_a_steps_layers_leave_its_rows():
    pool = small_pool(n_pages=8)
    x = torch.randn((2, 2, 2, 8), device="cuda")
    seqs, starts = dev([0, 2]), None
    pool.append(x[0], x[0], seqs, starts, layer=0)
    pool.fork(dev([0]), dev([2]))                               # not empty
    refused(pool, "index")
    pool.free(dev([0, 9]))                                      # no such sequence
    refused(pool, "index")
    pool.append(x[1], x[1], seqs, starts, layer=1)
    pool.check()
    for i, (s, pos) in enumerate(((0, 6), (2, 7))):
        page = int(pool.table[s, pos // 4])
        for layer in range(2):
            assert torch.equal(pool.k[layer, page, :, pos % 4], x[layer, i]) and torch.equal(pool.v[layer, page, :, pos % 4], x[layer, i])


# -- bookkeeping that does not agree with itself -------------------------------

def books(pool):
    return [t.clone() for t in (pool.refs, pool.lens, pool.table, pool.k, pool.v)]


def unchanged(pool, before):
    return all(torch.equal(a, b) for a, b in zip(before, books(pool)))


@pytest.mark.parametrize("compact", [False, True])
@pytest.mark.parametrize("wrong", ["page outside", "page below", "count of one page", "count of a shared page"])
def test_a_free_that_cannot_be_done_whole_changes_nothing(wrong, compact):
    pool = small_pool(n_pages=12)
    pool.fork(dev([0, 2]), dev([3, 4]))
    pool.free(dev([2]))                     # a hole before the last pages
    pool.check()
    if wrong == "page outside":
        pool.table[4, 1] = pool.n_pages
    elif wrong == "page below":
        pool.table[0, 0] = -3
    elif wrong == "count of one page":
        pool.refs[int(pool.table[4, 1])] = 0
    else:
        pool.refs[int(pool.table[0, 0])] = 1    # two sequences hold it
    before = books(pool)
    pool.free(dev([0, 3, 4, 3]), compact=compact)
    refused(pool, "outside the pool" if wrong.startswith("page") else "inconsistent")
    assert unchanged(pool, before)


def test_a_fork_of_pages_that_nobody_holds_is_refused():
    for col, rows in ((0, 6), (1, 6), (0, 4)):
        pool = small_pool(n_pages=12)
        pool.refs[int(pool.table[0, col])] = 0
        before = books(pool)
        pool.fork(dev([0, 2]), dev([3, 4]), dev([rows, 7]))
        refused(pool, "inconsistent")
        assert unchanged(pool, before)


def test_a_compaction_reports_and_leaves_entries_of_pages_that_nobody_holds():
    pool = small_pool(n_pages=12)
    x = torch.randn((2, 2, 8, 2, 8), device="cuda")
    pool.append(x[0], x[1], dev([1, 3]), dev([0, 4, 8]))     # pages 4 and 5
    pool.append(x[0, :, :4], x[1, :, :4], dev([4]), dev([0, 4]))  # page 6
    pool.free(dev([0]))                                      # pages 0 and 1 are holes; 2 .. 6 held
    pool.check()
    assert pool.table[[1, 3, 4], 0].tolist() == [4, 5, 6]
    pool.refs[5] = 0                                         # sequence 3's page counts as free: 4 are held, 4 and 6 move
    pool.table[2, 1] = 0                                     # and sequence 2 names a hole
    pool._scratch[8:].fill_(7)                               # what earlier calls may have left
    pool.free(compact=True)
    refused(pool, "inconsistent")
    assert pool.table[[1, 3, 4], 0].tolist() == [0, 5, 1] and pool.table[2, :2].tolist() == [2, 0]
    assert pool.refs.tolist() == [1, 1, 1, 1] + [0] * 8
    assert torch.equal(pool.k[:, 0], x[0, :, :4].transpose(1, 2)) and torch.equal(pool.v[:, 1], x[1, :, :4].transpose(1, 2))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("H,kv,hs,members,n", [(32, 8, 64, 32, 16384), (16, 16, 128, 40, 8192)])
def test_keys_that_all_lie_in_whole_tensor_core_tiles(dtype, H, kv, hs, members, n):
    """Attention right after a fork of a long prompt: no key is left for the walk."""
    groups = [(n, members)]
    lens = np.full(members, n)
    pool, rows, args = grouped(dtype, groups, lens, kv, hs, 64, seed=n)
    q = torch.randn((members, H, hs), device="cuda").to(DT[dtype])
    lse = torch.empty((members, H), device="cuda")
    out = pool.attention(q, 0, lse=lse, **args)
    pool.check()
    check_wide(out, lse, q, rows, dtype, 1 / math.sqrt(hs), [0, members // 2, members - 1])


# -- pools with room for long sequences ----------------------------------------

@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,shared", [(200, False), (160, True), (1024, False), (1024, True)])
def test_many_rows_of_a_pool_with_room_for_long_sequences(dtype, B, shared):
    """What a call may do hangs on what its sequences hold, not on what their tables could hold."""
    H = kv = 32
    ps, max_pages = 128, 1024
    rng = np.random.default_rng(B)
    prefix = 128 * 9 if shared else 0
    lens = prefix + rng.integers(0, 200, B)
    groups = [(prefix, B // 4), (prefix, B - B // 4)] if shared else [(0, 1)] * B
    small, rows, args = grouped(dtype, groups, lens, kv, 8, ps, seed=B)
    table = torch.zeros((B, max_pages), dtype=torch.int32, device="cuda")
    table[:, :small.max_pages] = small.table
    pool = pkg.PagePool.from_tensors(small.k, small.v, small.refs, small.lens, table)
    q = torch.randn((B, H, 8), device="cuda").to(DT[dtype])
    lse = torch.empty((B, H), device="cuda")
    out = pool.attention(q, 0, lse=lse, **(args if shared else {}))
    pool.check()
    check_wide(out, lse, q, rows, dtype, 1 / math.sqrt(8), sorted({0, B // 4, B - 1, *rng.integers(0, B, 10).tolist()}))
    assert torch.equal(out, small.attention(q, 0, **(args if shared else {})))
    # sequences that hold too much together: refused, the output as it was
    kept = out.clone()
    pool.lens.fill_(ps * max_pages)
    if B == 1024 and not shared:
        wide = pkg.PagePool.from_tensors(small.k, small.v, small.refs, pool.lens, torch.zeros((B, 8 * max_pages), dtype=torch.int32, device="cuda"))
        pool.lens.fill_(8 * ps * max_pages)
        wide.attention(q, 0, out=out)
        with pytest.raises(pkg.L2Error, match="index"):
            wide.check()
        wide.attention(q, 0, out=out, group_starts=dev([0, 1024]), prefix_lens=dev([7]))
        with pytest.raises(pkg.L2Error, match="index"):
            wide.check()
        assert torch.equal(out, kept)


def test_rows_read_into_shared_memory_are_refused():
    pool = small_pool()
    flat = torch.zeros(4096, device="cuda")
    for strides in ((8, 8, 1), (16, 0, 1), (24, 32, 1)):   # rows over heads, heads over one another, half over one another
        t = flat.as_strided((5, 2, 8), strides)
        with pytest.raises(pkg.L2Error, match="overlap"):
            pool.read(t, t, dev([0]), dev([0, 5]), layer=0)
    with pytest.raises(pkg.L2Error, match="same memory"):
        k = flat.as_strided((1, 4, 2, 4, 8), (0, 64, 8, 8, 1))
        pkg.PagePool.from_tensors(k, k, dev(np.zeros(4)), dev(np.zeros(2)), dev(np.zeros((2, 4))))
    for strides in ((16, 8, 1), (8, 40, 1), (24, 8, 1)):
        k, v = (torch.zeros(4096, device="cuda").as_strided((5, 2, 8), strides) for _ in range(2))
        pool.read(k, v, dev([0]), dev([0, 5]), layer=1)
        page = pool.table[0, :2].long()
        assert torch.equal(k, pool.k[1, page].transpose(1, 2).reshape(8, 2, 8)[:5]) and torch.equal(v, pool.v[1, page].transpose(1, 2).reshape(8, 2, 8)[:5])
    pool.check()


@pytest.mark.parametrize("starts", [None, [0, 3, 4]])
def test_rows_without_an_extension_do_not_go_into_pages_that_others_hold(starts):
    pool = pkg.PagePool(2, 12, 2, 4, 8, 6, 4)
    x = torch.randn((2, 13, 2, 8), device="cuda")
    pool.append(x, x, dev([0, 2]), dev([0, 8, 13]))      # two full pages; a full one and a row
    pool.fork(dev([0]), dev([1]))                        # shares both
    pool.check()
    k, v = pool.k.clone(), pool.v.clone()
    n = 2 if starts is None else starts[-1]
    y = torch.randn((n, 2, 8), device="cuda")
    pool.append(y, y, dev([1, 2]), None if starts is None else dev(starts), layer=1, extend=False)
    refused(pool, "index")
    page = int(pool.table[2, 1])
    k[1, page, :, 0], v[1, page, :, 0] = y[-1], y[-1]    # sequence 2's own page takes its row
    assert torch.equal(pool.k, k) and torch.equal(pool.v, v)
    pool.free(dev([0]))                                  # now they are sequence 1's alone
    pool.append(y, y, dev([1, 2]), None if starts is None else dev(starts), layer=1, extend=False)
    pool.check()
    at = n - 1
    page = int(pool.table[1, 1])
    assert torch.equal(pool.k[1, page, :, 4 - at:], y[:at].transpose(0, 1))


@pytest.mark.parametrize("H,members,prefix", [(1, 1, 0), (8, 1, 0), (12, 1, 0), (16, 1, 0), (1, 11, 60), (4, 40, 4096)])
@pytest.mark.parametrize("hs", [32, 64, 128])
def test_a_large_value_of_v_does_not_round_to_infinity(H, members, prefix, hs):
    """fp32: one key has all the weight (the others' is below 2^-150, so 0) and a V up to 2^-20 below the largest float; the
    other keys' V is of normal size, so that the sums, which are fp32, stay finite however many weights of 1 a part begins with.
    The tensor-core role takes weights as 2^fma(score, c, -m) with m = round(score c), so the largest is not 1 but up to
    2^(half a step of m) <= 1 + 2^-17 for m below 256: V has to be that much smaller for its product to be finite, 2^-16 here."""
    groups = [(prefix, members)]
    pool, rows, args = grouped("fp32", groups, np.full(members, prefix + 50), 1, hs, 16, seed=hs)
    top = float(np.finfo(np.float32).max) * (1 - 2.0 ** (-16 if prefix >= 4096 else -20))
    pool.k.zero_()
    at = prefix // 2 if prefix else 17
    for b in range(members):
        pool.k[0, int(pool.table[b, at // 16]), 0, at % 16, 0] = 1.0
    v = (torch.rand(hs, device="cuda") * 2 - 1) * top
    v[::2], v[1::4] = top, -top
    pool.v[0, int(pool.table[0, at // 16]), 0, at % 16] = v
    q = torch.zeros((members, H, hs), device="cuda")
    q[..., 0] = 120.0
    out = pool.attention(q, 0, scale=1.0, **(args if members > 1 else {}))
    pool.check()
    want = rows(0)[1][at, 0]
    # weight and sum of weights are one number: what is left are the halves, 2^-22 of the value, and a rounding or two
    assert float(((out[0].double() - want) / want).abs().max()) <= 2.0 ** -21


@pytest.mark.parametrize("hs", [64, 128])
def test_infinite_keys_give_the_same_bits_every_time(hs):
    """fp32 prefixes on the tensor cores: tiles with infinities are summed again, by two warps over the same scores."""
    members, n, H = 40, 6400, 8
    pool, rows, args = grouped("fp32", [(n, members)], np.full(members, n) + np.arange(members) % 3, 2, hs, 64, seed=hs)
    q = torch.randn((members, H, hs), device="cuda")
    q[..., 3] = q[..., 3].abs() + 0.5
    gone = torch.zeros(n + 64, dtype=torch.bool, device="cuda")
    for j in range(0, n // 64, 2):
        page = int(pool.table[0, j])
        pool.k[0, page, :, (j * 7) % 64, 3] = -math.inf
        gone[64 * j + (j * 7) % 64] = True
    lse = torch.empty((members, H), device="cuda")
    out = pool.attention(q, 0, lse=lse, **args)
    pool.check()

    def visible(b):
        k, v = rows(b)
        return k[~gone[:len(k)]], v[~gone[:len(k)]]
    check_wide(out, lse, q, visible, "fp32", 1 / math.sqrt(hs), [0, 1, members - 1])
    again = torch.empty_like(lse)
    for _ in range(30):
        assert torch.equal(pool.attention(q, 0, lse=again, **args), out) and torch.equal(again, lse)
    pool.check()


def test_one_layers_rows_do_not_go_to_every_layer():
    pool = small_pool()
    x = torch.randn((2, 2, 8), device="cuda")
    before = books(pool)
    for layer in (-1, -2, 2):
        for call in (lambda: pool.append(x, x, dev([0, 2]), layer=layer), lambda: pool.append(x, x, dev([0, 2]), layer=layer, extend=True),  # noqa: B023
                     lambda: pool.read(x, x, dev([0, 2]), layer=layer)):  # noqa: B023
            with pytest.raises((ValueError, pkg.L2Error)):
                call()
    pool.check()
    assert unchanged(pool, before)


def test_scales_that_fp32_does_not_hold_are_refused():
    pool = small_pool()
    q = torch.zeros((1, 2, 8), device="cuda")
    for scale in (2.4e38, -3e38, 1e39, -1e300):     # times log2(e): above 3.4e38
        with pytest.raises(pkg.L2Error, match="finite"):
            pool.attention(q, 0, scale=scale)
    for scale in (2.3e38, -2.3e38, 1e-300, 0.0):    # all scores 0: the mean of the rows
        out = pool.attention(q, 0, scale=scale)
        pool.check()
        page = pool.table[0, :2].long()
        want = pool.v[0, page].double().transpose(1, 2).reshape(8, 2, 8)[:6]
        # six weights of 1: five adds of a step each, the product with 1 / 6, the output
        assert bool(((out[0].double() - want.mean(0)).abs() <= 8 * 2.0 ** -23 * want.abs().mean(0)).all())


def test_arguments_of_a_call_on_another_stream_may_be_dropped():
    """The calls wait behind a long kernel of their stream while the memory of their arguments would be handed out again."""
    pool = pkg.PagePool(1, 40, 2, 16, 64, 6, 8)
    side = torch.cuda.Stream()
    k, v = (torch.randn((1, 300, 2, 64), device="cuda") for _ in range(2))
    q = torch.randn((3, 4, 64), device="cuda")
    keep, lens = (k.clone(), v.clone(), q.clone()), [100, 93, 107]
    index = dev([0, 1, 2]), dev([0, 100, 193, 300]), dev([0, 1, 2]), dev([3, 4, 5]), dev([64, 64, 64]), dev([0, 3]), dev([0])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(60_000_000)
    pool.append(k, v, index[0], index[1], stream=side)
    pool.fork(index[2], index[3], index[4], stream=side)
    lse = torch.empty((3, 4), device="cuda")
    out = pool.attention(q, 0, seqs=index[3], group_starts=index[5], prefix_lens=index[6], lse=lse, stream=side)
    rows_k, rows_v = (torch.zeros((100, 2, 64), device="cuda") for _ in range(2))
    del k, v, q, index
    junk = [torch.full(n, -99, dtype=torch.int32, device="cuda") for n in ((1, 300, 2, 64),) * 4 + ((3, 4, 64),) * 4 + ((3,), (2,), (4,), (1,)) * 64]
    torch.cuda.synchronize()
    pool.check()
    assert pool.lens.tolist() == lens + [64, 64, 64] and len(junk) == 264
    pool.read(rows_k, rows_v, dev([0]), dev([0, 100]), layer=0)
    assert torch.equal(rows_k, keep[0][0, :100]) and torch.equal(rows_v, keep[1][0, :100])
    again = pool.attention(keep[2], 0, seqs=dev([3, 4, 5]), group_starts=dev([0, 3]), prefix_lens=dev([0]))
    assert torch.equal(out, again) and bool(lse.isfinite().all())
