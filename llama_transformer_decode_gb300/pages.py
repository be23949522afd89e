"""Paged KV cache: a pool of pages that sequences take as they grow and share
after a fork, and decode attention over it (``l2_pages_*`` of ``include/l2.h``).

Like the rest of the binding this only marshals arguments: rows are moved, and
counts, lengths and tables changed, by the CUDA kernels.  Calls enqueue on
``stream`` (default: torch's current stream), never wait, and can be captured
into a CUDA graph.
"""
from __future__ import annotations

import ctypes
import math

from . import _native
from ._native import L2Pages, L2PagesAttention, L2PagesRows

L2_F32, L2_BF16, L2_F16 = 0, 1, 2
L2_PAGES_TIMEOUT, L2_PAGES_BAD_PAGE, L2_PAGES_BAD_CALL, L2_PAGES_FULL = 1, 2, 4, 8
_REASONS = ((L2_PAGES_TIMEOUT, "a kernel's bounded wait ran out"),
            (L2_PAGES_BAD_PAGE, "a table entry outside the pool"),
            (L2_PAGES_BAD_CALL, "bad index arrays or inconsistent bookkeeping"),
            (L2_PAGES_FULL, "too few free pages"))
_L2_EDEVICE, _L2_ETIMEOUT = -5, -6


def _raise(code: int):
    from . import L2Error
    raise L2Error(code, _native.load().l2_last_error(None).decode())


class PagePool:
    """A pool of ``n_pages`` pages of ``page_size`` rows per layer, for ``n_seqs``
    sequences of at most ``max_pages`` pages.

    ``k``, ``v``: [n_layers][n_pages][n_kv_heads][page_size][head_size] CUDA tensors
    (float32, bfloat16 or float16; other orders in memory as strided views);
    ``refs`` [n_pages], ``lens`` [n_seqs], ``table`` [n_seqs][max_pages]: int32.
    """

    def __init__(self, n_layers: int, n_pages: int, n_kv_heads: int, page_size: int, head_size: int, n_seqs: int,
                 max_pages: int, dtype=None, device="cuda"):
        import torch
        dtype = dtype if dtype is not None else torch.float32
        shape = (n_layers, n_pages, n_kv_heads, page_size, head_size)
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)  # noqa: E731
        self._bind(torch.zeros(shape, dtype=dtype, device=device), torch.zeros(shape, dtype=dtype, device=device),
                   ints(n_pages), ints(n_seqs), ints(n_seqs, max_pages))

    @classmethod
    def from_tensors(cls, k, v, refs, lens, table) -> "PagePool":
        """A pool over tensors the caller keeps (and may share with its own code)."""
        self = cls.__new__(cls)
        self._bind(k, v, refs, lens, table)
        return self

    def _bind(self, k, v, refs, lens, table):
        import torch
        kinds = {torch.float32: L2_F32, torch.bfloat16: L2_BF16, torch.float16: L2_F16}
        if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be alike, [layers][pages][kv heads][rows][head size]")
        if k.dtype not in kinds:
            raise ValueError("k and v must be float32, bfloat16 or float16")
        if k.shape[4] > 1 and k.stride(4) != 1:
            raise ValueError("the last dimension of k and v must be contiguous")
        for name, t, shape in (("refs", refs, (k.shape[1],)), ("lens", lens, None), ("table", table, None)):
            if t.dtype != torch.int32 or not t.is_contiguous() or t.device != k.device or (shape and tuple(t.shape) != shape):
                raise ValueError(f"{name} must be a contiguous int32 tensor of the pool's device and size")
        if lens.dim() != 1 or table.dim() != 2 or table.shape[0] != lens.shape[0]:
            raise ValueError("lens must be [sequences] and table [sequences][pages]")
        if not k.is_cuda:
            raise ValueError("expected CUDA tensors")
        self.k, self.v, self.refs, self.lens, self.table = k, v, refs, lens, table
        self.dtype, self.device = k.dtype, k.device
        self.n_layers, self.n_pages, self.n_kv_heads, self.page_size, self.head_size = k.shape
        self.n_seqs, self.max_pages = table.shape
        self._lib = _native.load()
        ints = torch.zeros(64 + self._lib.l2_pages_scratch_ints(self.n_pages), dtype=torch.int32, device=k.device)
        self.status, self._scratch = ints[:1], ints[64:]
        self._c = L2Pages(k.data_ptr(), v.data_ptr(), refs.data_ptr(), lens.data_ptr(), table.data_ptr(),
                          self.status.data_ptr(), self._scratch.data_ptr(), *k.stride()[:4], kinds[k.dtype], *k.shape,
                          *table.shape)
        self._ref = ctypes.byref(self._c)
        rc = self._lib.l2_pages_init(self._ref)
        if rc:
            _raise(rc)
        self._ws = {}  # workspace bytes per (rows, groups, heads)
        self._torch, self._int32, self._index = torch, torch.int32, k.get_device()
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._scale = 1.0 / math.sqrt(self.head_size)
        self._bytes = torch.empty(0, dtype=torch.uint8, device=k.device)  # workspaces are made like it

    # -- helpers -------------------------------------------------------------
    def _stream(self, stream):
        return self._raw_stream(self._index) if stream is None else stream.cuda_stream

    def _ints(self, name, t, n=None):
        """Address of an index array; n: its length, where the call fixes it."""
        if not isinstance(t, self._torch.Tensor) or t.dtype is not self._int32 or t.get_device() != self._index or t.dim() != 1 \
                or not t.is_contiguous() or (n is not None and t.numel() != n):
            raise ValueError(f"{name} must be a contiguous int32 tensor [{'n' if n is None else n}] on {self.device}")
        return t.data_ptr()

    def _rows(self, name, t, dims):
        """Address, shape and strides of a tensor of rows of head_size."""
        shape, st = t.shape, t.stride()
        if t.dtype is not self.dtype or t.get_device() != self._index or len(shape) != dims or shape[-1] != self.head_size \
                or (st[-1] != 1 and shape[-1] > 1):
            raise ValueError(f"{name} must have {dims} dimensions, the pool's type, device and head size, its last one contiguous")
        return t.data_ptr(), shape, st

    @staticmethod
    def _used_on(stream, *tensors):
        """A call on a stream of its own may run after its arguments are dropped: their memory is kept until it has."""
        if stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def check(self):
        """Waits for the pool's device and raises L2Error if a call could not be done (and clears the status)."""
        self._torch.cuda.synchronize(self.device)
        bits = int(self.status.item())
        if bits:
            from . import L2Error
            self.status.zero_()
            raise L2Error(_L2_ETIMEOUT if bits & L2_PAGES_TIMEOUT else _L2_EDEVICE, "page pool: " + "; ".join(text for bit, text in _REASONS if bits & bit))

    # -- API -----------------------------------------------------------------
    def append(self, k, v, seqs, starts=None, layer=None, extend=None, stream=None):
        """Rows ``k``, ``v`` ([rows][kv heads][head size] of ``layer``, or with a leading
        dimension of all layers) at the ends of sequences ``seqs``: rows
        starts[i]..starts[i + 1] - 1 go to seqs[i] (row i, without ``starts``).  ``extend``
        (default: with all layers, or layer 0) first lengthens the sequences."""
        a = self._moved(k, v, seqs, starts, layer, (layer is None or layer == 0) if extend is None else bool(extend))
        rc = self._lib.l2_pages_append(self._ref, ctypes.byref(a), self._stream(stream))
        if rc:
            _raise(rc)
        self._used_on(stream, k, v, seqs, starts)

    def read(self, k, v, seqs, starts=None, layer=None, stream=None):
        """Into ``k``, ``v`` (shaped as for append): rows starts[i]..starts[i + 1]-1 receive the first rows of seqs[i]."""
        a = self._moved(k, v, seqs, starts, layer, False)
        rc = self._lib.l2_pages_read(self._ref, ctypes.byref(a), self._stream(stream))
        if rc:
            _raise(rc)
        self._used_on(stream, k, v, seqs, starts)

    def _moved(self, k, v, seqs, starts, layer, extend):
        whole = layer is None
        kp, shape, st = self._rows("k", k, 4 if whole else 3)
        vp, v_shape, v_st = self._rows("v", v, 4 if whole else 3)
        if shape != v_shape or st != v_st or shape[-2] != self.n_kv_heads or (whole and shape[0] != self.n_layers):
            raise ValueError("k and v must be alike, with the pool's layers and heads")
        if not whole and not 0 <= layer < self.n_layers:  # the library's -1 means every layer, whose rows have a leading dimension
            raise ValueError(f"layer {layer} outside 0..{self.n_layers - 1}")
        n = len(seqs)
        return L2PagesRows(n, shape[-3], self._ints("seqs", seqs), None if starts is None else self._ints("starts", starts, n + 1),
                           -1 if whole else int(layer), int(extend), kp, vp, st[0] if whole else 0, st[-3], st[-2])

    def fork(self, src, dst, rows=None, stream=None):
        """Empty sequence dst[i] becomes the first rows[i] rows of src[i] (all, without ``rows``)."""
        n = len(src)
        rc = self._lib.l2_pages_fork(self._ref, n, self._ints("src", src, n), self._ints("dst", dst, n),
                                     None if rows is None else self._ints("rows", rows, n), self._stream(stream))
        if rc:
            _raise(rc)
        self._used_on(stream, src, dst, rows)

    def free(self, seqs=None, compact=False, stream=None):
        """Empties sequences ``seqs`` and gives their pages back; ``compact`` then closes the pool up."""
        n = 0 if seqs is None else len(seqs)
        rc = self._lib.l2_pages_free(self._ref, n, self._ints("seqs", seqs) if n else None, int(bool(compact)),
                                     self._stream(stream))
        if rc:
            _raise(rc)
        self._used_on(stream, seqs)

    def attention(self, q, layer: int, seqs=None, group_starts=None, prefix_lens=None, scale=None, out=None, lse=None,
                  stream=None):
        """Attention of ``q`` [rows][heads][head size], row b over all cached rows of
        sequence seqs[b] (b, without ``seqs``), with prefixes shared by groups of rows read
        once (``l2_pages_attention``).  ``lse``: a float32 [rows][heads] tensor for the log
        sums, or None.  Returns ``out``."""
        qp, (B, H, _), q_st = self._rows("q", q, 3)
        G = gs = pl = 0
        if group_starts is not None:
            G = len(group_starts) - 1
            if G < 1 or prefix_lens is None:
                raise ValueError("group_starts needs at least one group, and prefix_lens")
            gs, pl = self._ints("group_starts", group_starts), self._ints("prefix_lens", prefix_lens, G)
        elif prefix_lens is not None:
            raise ValueError("prefix_lens needs group_starts")
        need = self._ws.get((B, G, H))
        if need is None:
            need = self._lib.l2_pages_attention_ws(self._ref, B, G, H)
            if need < 0:
                _raise(int(need))
            self._ws[(B, G, H)] = need
        torch = self._torch
        fresh = out is None
        if stream is None:
            if fresh:
                out = torch.empty((B, H, self.head_size), dtype=self.dtype, device=self.device)
            ws = self._bytes.new_empty(need)
        else:  # the workspace belongs to the stream that uses it
            with torch.cuda.stream(stream):
                if fresh:
                    out = torch.empty((B, H, self.head_size), dtype=self.dtype, device=self.device)
                ws = self._bytes.new_empty(need)
        if fresh:
            op, o_row, o_head = out.data_ptr(), H * self.head_size, self.head_size
        else:
            op, o_shape, (o_row, o_head, _) = self._rows("out", out, 3)
            if o_shape != q.shape:
                raise ValueError("out must have q's shape")
        if lse is not None and (lse.dtype is not torch.float32 or lse.get_device() != self._index or not lse.is_contiguous()
                                or tuple(lse.shape) != (B, H)):
            raise ValueError("lse must be a contiguous float32 tensor [rows][heads] of the pool's device")
        a = L2PagesAttention(int(layer), B, G, H, qp, op, None if lse is None else lse.data_ptr(),
                             None if seqs is None else self._ints("seqs", seqs, B), gs, pl, q_st[0], q_st[1], o_row, o_head,
                             self._scale if scale is None else float(scale))
        rc = self._lib.l2_pages_attention(self._ref, ctypes.byref(a), ws.data_ptr(), need, self._stream(stream))
        if rc:
            _raise(rc)
        self._used_on(stream, q, seqs, group_starts, prefix_lens, None if fresh else out, lse)
        return out
