"""Pools whose strides give two rows the same memory are refused when they are made; every order of dimensions that keeps
them apart is not.  Host-only."""
import ctypes
import itertools

import pytest

import llama_transformer_decode_gb300 as pkg
from tests.test_pages_host import lib, pool_struct, text  # noqa: F401

SIZES = dict(n_layers=2, n_pages=4, n_kv_heads=2, page_size=4)
NAMES = ("layer_stride", "page_stride", "head_stride", "row_stride")


def said(lib, **strides):  # noqa: F811
    assert lib.l2_pages_init(ctypes.byref(pool_struct(**SIZES, **strides))) == pkg.L2_EINVAL  # host memory at the latest
    return text(lib)


@pytest.mark.parametrize("bad", [
    dict(row_stride=64, head_stride=64, page_stride=1024, layer_stride=4096),     # a row of one head is another's
    dict(row_stride=64, head_stride=192, page_stride=1024, layer_stride=4096),    # heads start inside the rows before
    dict(row_stride=64, head_stride=256, page_stride=448, layer_stride=4096),     # pages over one another
    dict(row_stride=64, head_stride=256, page_stride=512, layer_stride=512),      # layers over one another
    dict(row_stride=64, head_stride=256, page_stride=1 << 40, layer_stride=1 << 40)])
def test_rows_that_share_memory(lib, bad):  # noqa: F811
    assert "same memory" in said(lib, **bad)


def test_every_order_of_dimensions(lib):  # noqa: F811
    for order in itertools.permutations(range(4)):
        for gap in (0, 8):
            strides, span = {}, 64 + gap
            for d in order:
                strides[NAMES[d]] = span
                span = span * (2, 4, 2, 4)[d] + gap
            assert "device memory" in said(lib, **strides), (order, strides)


def test_dimensions_of_one_index_have_no_stride(lib):  # noqa: F811
    p = pool_struct(n_layers=1, n_pages=1, n_kv_heads=1, page_size=4, layer_stride=0, page_stride=-5, head_stride=64, row_stride=64)
    assert lib.l2_pages_init(ctypes.byref(p)) == pkg.L2_EINVAL and "device memory" in text(lib)
