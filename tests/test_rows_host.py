"""The entry points on rows of a caller's own layer code (rotary positions, rules on logits) and those on drafted tokens
refuse what the host can see, before anything is enqueued.  Host-only."""
import ctypes
import math

import numpy as np
import pytest

import llama_transformer_decode_gb300 as pkg
from llama_transformer_decode_gb300 import _native
from tests import tree_ref
from tests.test_pages_host import pool_struct

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    try:
        return _native.load()
    except OSError as e:
        pytest.skip(f"cannot load the CUDA runtime here: {e}")


def text(lib):
    return lib.l2_last_error(None).decode()


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(_native.L2PagesTreeAttention) == 16 + 6 * 8 + 4 * 8 + 8
    assert ctypes.sizeof(_native.L2PagesAccept) == 8 + 8 * 8
    assert ctypes.sizeof(_native.L2RopePlan) == 16 + 128 * 8
    assert ctypes.sizeof(_native.L2RopeRows) == 24 + 5 * 8 + 8 * 8
    assert ctypes.sizeof(_native.L2TokenRules) == 16 + 8 + 10 * 8 + 8
    assert ctypes.sizeof(_native.L2TokenRows) == 8 + 6 * 8 + 8 + 2 * 8 + 2 * 8 + 8 + 8


def test_calls_on_trees_need_a_pool_and_arguments(lib):
    bare = pool_struct()
    for pool in (None, ctypes.byref(bare)):
        assert lib.l2_pages_tree_attention_ws(pool, 1, 1, 2) == pkg.L2_EINVAL
        assert lib.l2_pages_tree_attention(pool, ctypes.byref(_native.L2PagesTreeAttention()), None, 0, None) == pkg.L2_EINVAL
        assert lib.l2_pages_accept(pool, ctypes.byref(_native.L2PagesAccept(n=1)), None) == pkg.L2_EINVAL
        assert lib.l2_pages_keep(pool, ctypes.byref(_native.L2PagesAccept(n=1)), None) == pkg.L2_EINVAL
    assert "l2_pages_init" in text(lib)
    # a pool that passes for initialised (device 0): what comes after is refused by itself, before any device is asked
    ready = pool_struct(ready=0x50a6e500)
    p = ctypes.byref(ready)
    for call, args in ((lib.l2_pages_tree_attention, (None, None, 0, None)), (lib.l2_pages_accept, (None, None)), (lib.l2_pages_keep, (None, None))):
        assert call(p, *args) == pkg.L2_EINVAL
        assert "NULL" in text(lib)
    A = _native.L2PagesTreeAttention
    for bad, word in ((dict(n=0, rows=1, n_heads=2), "n = 0"), (dict(n=1025, rows=1, n_heads=2), "n = 1025"), (dict(n=1, rows=0, n_heads=2), "outside 1..1024"),
                      (dict(n=1, rows=1025, n_heads=2), "outside 1..1024"), (dict(n=1, rows=1, n_heads=1), "n_heads"), (dict(n=1, rows=1, n_heads=1025), "n_heads"),
                      (dict(n=1, rows=1, n_heads=2, layer=2), "layer"), (dict(n=1, rows=1, n_heads=2, layer=-1), "layer"),
                      (dict(n=1, rows=1, n_heads=2, scale=math.nan), "scale"), (dict(n=1, rows=1, n_heads=2, scale=1e39), "scale"),
                      (dict(n=1, rows=2, n_heads=2, q_row_stride=6), "q_row_stride"), (dict(n=1, rows=2, n_heads=2, out_row_stride=-64), "out_row_stride"),
                      (dict(n=1, rows=2, n_heads=2, out_row_stride=64, out_head_stride=64), "overlap"),
                      (dict(n=1, rows=1, n_heads=2, out_head_stride=64), "q is NULL")):
        assert lib.l2_pages_tree_attention(p, ctypes.byref(A(**{"scale": 1.0, **bad})), None, 0, None) == pkg.L2_EINVAL, bad
        assert word in text(lib), (bad, text(lib))
    C = _native.L2PagesAccept
    for call in (lib.l2_pages_accept, lib.l2_pages_keep):
        for bad, word in ((dict(n=0), "n = 0"), (dict(n=1025), "n = 1025"), (dict(n=1, rows=-1), "rows"), (dict(n=1, rows=65537), "rows"), (dict(n=1, rows=1), "seqs")):
            assert call(p, ctypes.byref(C(**bad)), None) == pkg.L2_EINVAL
            assert word in text(lib), (bad, text(lib))


def test_frequencies_and_plans(lib):
    f = (ctypes.c_double * 128)()
    for bad, word in (((0, 1e4, 0, 1, 0, 0, 0), "rot_dim"), ((3, 1e4, 0, 1, 0, 0, 0), "rot_dim"), ((258, 1e4, 0, 1, 0, 0, 0), "rot_dim"),
                      ((8, 0, 0, 1, 0, 0, 0), "base"), ((8, math.inf, 0, 1, 0, 0, 0), "base"), ((8, 1e4, 4, 1, 0, 0, 0), "scaling"),
                      ((8, 1e4, -1, 1, 0, 0, 0), "scaling"), ((8, 1e4, 1, 0, 0, 0, 0), "factor"), ((8, 1e4, 2, math.nan, 0, 0, 0), "factor"),
                      ((8, 1e4, 3, 2, 0, 1, 4), "original_len"), ((8, 1e4, 3, 2, 100, 4, 4), "low below high"), ((8, 1e-300, 2, 1e-300, 0, 0, 0), "not finite")):
        assert lib.l2_rope_freqs(*bad, f) == pkg.L2_EINVAL, bad
        assert word in text(lib), (bad, text(lib))
    assert lib.l2_rope_freqs(8, 1e4, 0, 1, 0, 0, 0, None) == pkg.L2_EINVAL
    assert lib.l2_rope_freqs(8, 1e4, 0, 1, 0, 0, 0, f) == pkg.L2_OK
    assert np.allclose(list(f)[:4], [1, 0.1, 0.01, 0.001], rtol=1e-14)
    # a base-scaled set: the fastest pair stays, the slowest is slowed by the factor; two elements turn as before
    assert lib.l2_rope_freqs(8, 1e4, 2, 4, 0, 0, 0, f) == pkg.L2_OK and f[0] == 1 and math.isclose(f[3], 0.001 / 4, rel_tol=1e-13)
    assert lib.l2_rope_freqs(2, 1e4, 2, 4, 0, 0, 0, f) == pkg.L2_OK and f[0] == 1
    plan = _native.L2RopePlan()
    ok = (ctypes.c_double * 4)(1.0, -0.25, 2 * math.pi, 1e-12)
    for bad in ((0, 0, ok, 1.0), (8, 2, ok, 1.0), (8, 0, ok, math.inf), (8, 0, ok, 1e39), (8, 0, None, 1.0), (8, 0, (ctypes.c_double * 4)(1, 2, 3, math.nan), 1.0)):
        assert lib.l2_rope_plan(ctypes.byref(plan), *bad) == pkg.L2_EINVAL
        assert plan.ready == 0
    assert lib.l2_rope_plan(None, 8, 0, ok, 1.0) == pkg.L2_EINVAL
    assert lib.l2_rope_plan(ctypes.byref(plan), 8, 0, ok, 1.0) == pkg.L2_OK
    for i, x in enumerate(ok):   # a turn as a fraction of 2^64, whole turns left out
        turn = (x / (2 * math.pi)) % 1.0
        assert abs(plan.turns[i] / 2.0 ** 64 - turn) < 2.0 ** -52 or (turn > 0.5 and abs(plan.turns[i] / 2.0 ** 64 + 1 - turn) < 2.0 ** -52)
    # far positions land where 64 bits say: the frequency and its division by 2 pi round by 2^-53 each, as does the statement here, and the fraction
    # by half of 2^-64 a position
    for i, pos in ((0, 10 ** 6), (1, 2 ** 31 - 1), (3, -123456789)):
        turn = plan.turns[i] * pos % 2 ** 64 / 2.0 ** 64
        want = (pos * ok[i] / (2 * math.pi)) % 1.0
        assert min(abs(turn - want), 1 - abs(turn - want)) < 4 * 2.0 ** -53 * max(1.0, abs(pos * ok[i])) + abs(pos) * 2.0 ** -64
    R = _native.L2RopeRows
    r = ctypes.byref(plan)
    assert lib.l2_rope(None, ctypes.byref(R()), None) == pkg.L2_EINVAL and lib.l2_rope(r, None, None) == pkg.L2_EINVAL
    assert lib.l2_rope(ctypes.byref(_native.L2RopePlan()), ctypes.byref(R()), None) == pkg.L2_EINVAL and "l2_rope_plan" in text(lib)
    for bad, word in ((dict(dtype=3, head_size=8), "dtype"), (dict(rows=-1, head_size=8), "rows"), (dict(rows=1 << 24, head_size=8), "rows"),
                      (dict(head_size=7), "head_size"), (dict(head_size=257), "head_size"), (dict(rows=1, head_size=8), "positions")):
        assert lib.l2_rope(r, ctypes.byref(R(**bad)), None) == pkg.L2_EINVAL
        assert word in text(lib), (bad, text(lib))
    assert lib.l2_rope(r, ctypes.byref(R(rows=0, head_size=8)), None) == pkg.L2_OK   # nothing to do


def test_rules_and_their_rows(lib):
    N = _native.L2TokenRules
    buf = (ctypes.c_int * 64)()
    at = ctypes.addressof(buf)
    fine = dict(n_seqs=2, vocab_size=100, max_len=4, history_stride=4, history=at, lens=at)
    for bad, word in ((dict(n_seqs=0), "n_seqs"), (dict(vocab_size=0), "vocab_size"), (dict(vocab_size=(1 << 24) + 1), "vocab_size"), (dict(max_len=-1), "max_len"),
                      (dict(max_len=1 << 24), "max_len"), (dict(n_bias=-1), "n_bias"), (dict(history_stride=3), "history_stride"), (dict(history=None), "history"),
                      (dict(max_len=0, lens=None), "lens"), (dict(), "device memory"), (dict(lens=at + 2), "device memory")):
        c = N(**{**fine, **bad})
        assert lib.l2_token_rules_init(ctypes.byref(c)) == pkg.L2_EINVAL and c.ready == 0
        assert word in text(lib), (bad, text(lib))
    assert lib.l2_token_rules_init(None) == pkg.L2_EINVAL
    T = _native.L2TokenRows
    assert lib.l2_token_rules(None, ctypes.byref(T()), None) == pkg.L2_EINVAL
    bare = N(**fine)
    assert lib.l2_token_rules(ctypes.byref(bare), ctypes.byref(T(n=1, rows=1)), None) == pkg.L2_EINVAL and "l2_token_rules_init" in text(lib)
    bare.ready = 0x5201e500   # passes for initialised (device 0)
    r = ctypes.byref(bare)
    for bad, word in ((dict(n=0), "n = 0"), (dict(n=65536), "n = 65536"), (dict(rows=-1), "rows"), (dict(rows=2), "rows"), (dict(rows=65536, starts=at), "rows"),
                      (dict(n=3, rows=3), "exceeds"), (dict(dtype=5), "dtype"), (dict(dtype=0, out_dtype=1), "out_dtype"), (dict(dtype=1, out_dtype=2), "out_dtype"),
                      (dict(n=2, rows=2, row_stride=-1), "row_stride"), (dict(n=2, rows=2, row_stride=100, out_row_stride=99), "out_row_stride"),
                      (dict(masks=at), "n_masks"), (dict(masks=at, n_masks=2, mask_stride=3, mask_rows=at), "mask_stride"), (dict(), "logits is NULL")):
        assert lib.l2_token_rules(r, ctypes.byref(T(**{**dict(n=1, rows=1), **bad})), None) == pkg.L2_EINVAL, bad
        assert word in text(lib), (bad, text(lib))
    assert lib.l2_token_rules(r, ctypes.byref(T(n=1, rows=0, starts=at)), None) == pkg.L2_OK


def test_the_binding_refuses_host_tensors():
    x = torch.zeros((2, 3, 8))
    rope = pkg.Rope(8)
    with pytest.raises(ValueError):
        rope.apply(torch.zeros(2, dtype=torch.int32), x)
    with pytest.raises(ValueError):
        pkg.TokenRules(10, torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_the_plain_statements():
    assert tree_ref.line([-1, 0, 0, 1], 3) == [0, 1, 3] and tree_ref.chain(3) == [-1, 0, 1]
    # the lowest of two children that fit; a root that is not the first is never reached
    assert tree_ref.accepted([-1, 0, 0, 1, -1], [5, 7, 7, 1, 7], [7, 1, 9, 4, 4]) == ([0, 1, 3], 4)
    got = tree_ref.rules([2.0, -2.0, 1.0, 1.0], [0, 1, 0], 1, [2], 2.0, 0.5, 0.25, [(3, 9.0), (3, 1.0)], [True, True, True, False])
    assert got.tolist() == [1.0 - 0.75, -4.0 - 0.75, 0.5 - 0.75, -math.inf]
    x = np.arange(6.0).reshape(1, 1, 6)
    quarter = np.array([[math.pi / 2]])
    assert np.allclose(tree_ref.rope(x, quarter, 1.0, False), [[[-1, 0, 2, 3, 4, 5]]]) and np.allclose(tree_ref.rope(x, quarter, 2.0, True), [[[-2, 0, 2, 3, 4, 5]]])
