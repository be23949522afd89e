"""The paged-cache entry points refuse what the host can see, before anything is enqueued, and the plain
statement the GPU tests compare with holds its own invariants.  Host-only."""
import ctypes

import numpy as np
import pytest

import llama_transformer_decode_gb300 as pkg
from llama_transformer_decode_gb300 import _native
from tests import pages_ref

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    try:
        return _native.load()
    except OSError as e:
        pytest.skip(f"cannot load the CUDA runtime here: {e}")


def pool_struct(**kw):
    buf = (ctypes.c_byte * 4096)()
    at = (ctypes.addressof(buf) + 255) // 256 * 256
    d = dict(k=at, v=at, refs=at, lens=at, table=at, status=at, scratch=at, layer_stride=4096, page_stride=1024, head_stride=256,
             row_stride=64, dtype=0, n_layers=2, n_pages=4, n_kv_heads=2, page_size=4, head_size=64, n_seqs=3, max_pages=4)
    d.update(kw)
    p = _native.L2Pages(**d)
    p._keep = buf
    return p


def text(lib):
    return lib.l2_last_error(None).decode()


@pytest.mark.parametrize("bad,word", [
    (dict(dtype=3), "dtype"), (dict(n_pages=0), "positive"), (dict(head_size=0), "positive"), (dict(max_pages=-1), "positive"),
    (dict(head_size=136), "head_size"), (dict(head_size=6), "head_size"), (dict(dtype=1, head_size=12), "head_size"),
    (dict(row_stride=63), "row_stride"), (dict(row_stride=66), "row_stride"), (dict(page_stride=-64), "page_stride"),
    (dict(head_stride=0), "head_stride"), (dict(max_pages=1 << 30), "positions"), (dict(k=0), "k is NULL"),
    (dict(table=0), "NULL"), (dict(), "device memory")])
def test_pools_the_host_can_refuse(lib, bad, word):
    p = pool_struct(**bad)
    assert lib.l2_pages_init(ctypes.byref(p)) == pkg.L2_EINVAL
    assert word in text(lib), text(lib)
    # and a pool that was not initialised is refused by every call
    idx = ctypes.c_void_p(p.refs or p.k)
    for call in (lambda: lib.l2_pages_fork(ctypes.byref(p), 1, idx, idx, None, None),
                 lambda: lib.l2_pages_free(ctypes.byref(p), 1, idx, 0, None),
                 lambda: lib.l2_pages_append(ctypes.byref(p), ctypes.byref(_native.L2PagesRows(n=1, rows=1)), None),
                 lambda: lib.l2_pages_attention_ws(ctypes.byref(p), 1, 0, 2),
                 lambda: lib.l2_pages_attention(ctypes.byref(p), ctypes.byref(_native.L2PagesAttention()), None, 0, None)):
        assert call() == pkg.L2_EINVAL
        assert "l2_pages_init" in text(lib), text(lib)


def test_null_pools_and_sizes(lib):
    assert lib.l2_pages_init(None) == pkg.L2_EINVAL
    assert lib.l2_pages_fork(None, 1, None, None, None, None) == pkg.L2_EINVAL
    assert lib.l2_pages_free(None, 1, None, 0, None) == pkg.L2_EINVAL
    assert lib.l2_pages_append(None, None, None) == pkg.L2_EINVAL
    assert lib.l2_pages_attention(None, None, None, 0, None) == pkg.L2_EINVAL
    assert lib.l2_pages_scratch_ints(0) == pkg.L2_EINVAL
    assert lib.l2_pages_scratch_ints(100) >= 300


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(_native.L2Pages) == 7 * 8 + 4 * 8 + 8 * 4 + 8  # ready, padded
    assert ctypes.sizeof(_native.L2PagesRows) == 8 + 2 * 8 + 8 + 2 * 8 + 3 * 8
    assert ctypes.sizeof(_native.L2PagesAttention) == 16 + 6 * 8 + 4 * 8 + 8


def test_the_binding_refuses_host_tensors():
    k = torch.zeros((1, 2, 1, 4, 8))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkg.PagePool.from_tensors(k, k, i, i, torch.zeros((2, 3), dtype=torch.int32))
    with pytest.raises(ValueError):
        pkg.PagePool.from_tensors(k, k[..., :4], i, i, torch.zeros((2, 3), dtype=torch.int32))
    with pytest.raises(ValueError):
        pkg.PagePool.from_tensors(k.double(), k.double(), i, i, torch.zeros((2, 3), dtype=torch.int32))


def test_the_plain_statement_keeps_counts_and_tables_in_step():
    rng = np.random.default_rng(0)
    ref = pages_ref.RefPool(40, 4, 10, 8)
    for _ in range(300):
        op = rng.integers(0, 3)
        if op == 0:
            seqs = rng.permutation(10)[:rng.integers(1, 10)]
            ref.append(seqs, [int(c) for c in rng.integers(0, 6, len(seqs))])
        elif op == 1:
            empty, full = np.flatnonzero(ref.lens == 0), np.flatnonzero(ref.lens > 0)
            if len(empty) and len(full):
                ref.fork([int(rng.choice(full))], [int(empty[0])])
        else:
            ref.free(rng.permutation(10)[:2], compact=bool(rng.integers(0, 2)))
        count = np.zeros(40, int)
        for s in range(10):
            h = ref.held(s)
            assert len(set(ref.table[s, :h])) == h
            np.add.at(count, ref.table[s, :h], 1)
            if ref.lens[s] % 4:
                assert ref.refs[ref.table[s, h - 1]] == 1
        assert count.tolist() == ref.refs.tolist()


def test_reading_and_a_handles_rows_refuse_what_the_host_sees(lib):
    assert lib.l2_pages_read(None, None, None) == pkg.L2_EINVAL
    assert lib.l2_pages_read(ctypes.byref(pool_struct()), ctypes.byref(_native.L2PagesRows(n=1, rows=1)), None) == pkg.L2_EINVAL
    assert "l2_pages_init" in text(lib), text(lib)
    assert lib.l2_kv_to_pages(None, 0, None, None, None) == pkg.L2_EINVAL
    assert lib.l2_kv_from_pages(None, 0, 1, None, None, None) == pkg.L2_EINVAL
