"""Rotary positions of queries and keys (``l2_rope`` of ``include/l2.h``), for layer code
that keeps its keys in a ``PagePool``.

Arguments are marshalled here; cosines, sines and products are the CUDA kernel's.  Calls enqueue
on ``stream`` (default: torch's current stream), never wait, and can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes

from . import _native
from ._native import L2RopePlan, L2RopeRows

_LAYOUTS = {"interleaved": 0, "half": 1}
_SCALINGS = {None: 0, "linear": 1, "base": 2, "bands": 3}


def _raise(code: int):
    from . import L2Error
    raise L2Error(code, _native.load().l2_last_error(None).decode())


class Rope:
    """Turns the first ``rot_dim`` elements of each head by their row's position.

    ``layout``: pairs are neighbours ("interleaved", as in the decoder's steps) or rot_dim / 2 apart ("half").
    ``kind``: how frequencies base^(-2i / rot_dim) are scaled for long contexts: None, "linear" (``factor``), "base"
    (``factor``) or "bands" (``factor``, ``original_len``, ``low``, ``high``), see ``l2_rope_freqs``.  ``freqs``: a
    sequence of rot_dim / 2 frequencies of the caller's instead.  ``amplitude`` multiplies cosines and sines.
    """

    def __init__(self, rot_dim: int, base: float = 10000.0, layout: str = "interleaved", kind: str | None = None, factor: float = 1.0,
                 original_len: float = 0.0, low: float = 1.0, high: float = 4.0, amplitude: float = 1.0, freqs=None):
        import torch
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}")
        if kind not in _SCALINGS:
            raise ValueError("kind must be None, 'linear', 'base' or 'bands'")
        self._lib, self._torch = _native.load(), torch
        self._kinds = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        self._raw_stream, self._int32 = torch._C._cuda_getCurrentRawStream, torch.int32
        self.rot_dim, self.layout = int(rot_dim), layout
        n = max(self.rot_dim // 2, 1)
        if freqs is None:
            table = (ctypes.c_double * n)()
            rc = self._lib.l2_rope_freqs(self.rot_dim, float(base), _SCALINGS[kind], float(factor), float(original_len), float(low),
                                         float(high), table) if n <= _native.ROPE_MAX // 2 else 0
            if rc:
                _raise(rc)
        else:
            if kind is not None or len(freqs) != n:
                raise ValueError("freqs are rot_dim / 2 frequencies, without a kind of scaling")
            table = (ctypes.c_double * n)(*(float(f) for f in freqs))
        self._plan = L2RopePlan()
        self._ref = ctypes.byref(self._plan)
        rc = self._lib.l2_rope_plan(self._ref, self.rot_dim, _LAYOUTS[layout], table, float(amplitude))
        if rc:
            _raise(rc)
        self.freqs = list(table)

    def apply(self, positions, q=None, k=None, out_q=None, out_k=None, stream=None):
        """Turns ``q`` and ``k`` ([rows][heads][head size], float32, bfloat16 or float16, rows and heads at any strides) by
        ``positions`` (int32 [rows]).  Results go to ``out_q`` and ``out_k`` (in place: the tensor itself), by default new
        tensors.  Returns (out_q, out_k), None for one that is not given."""
        x = q if q is not None else k
        if x is None or (q is None and out_q is not None) or (k is None and out_k is not None):
            raise ValueError("q, k or both, and an output only for one that is given")
        kind, index, shape = self._kinds.get(x.dtype), x.get_device(), x.shape
        if kind is None or index < 0 or len(shape) != 3:
            raise ValueError("expected float32, bfloat16 or float16 CUDA tensors [rows][heads][head size]")
        rows, hs = shape[0], shape[2]
        if not isinstance(positions, self._torch.Tensor) or positions.dtype is not self._int32 or positions.get_device() != index \
                or positions.shape != (rows,) or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 tensor [{rows}] on the device of q and k")
        a = L2RopeRows(rows, kind, hs, 0, 0, positions.data_ptr())
        q_new, k_new = out_q is None, out_k is None
        if q is not None:
            s = self._side(q, x)
            if q_new:
                out_q = self._new(q, stream)
            o = self._side(out_q, q)
            if out_q.shape != q.shape:
                raise ValueError("an output must have its input's shape")
            a.n_heads, a.q, a.q_out = q.shape[1], q.data_ptr(), out_q.data_ptr()
            a.q_row_stride, a.q_head_stride, a.q_out_row_stride, a.q_out_head_stride = s[0], s[1], o[0], o[1]
        if k is not None:
            s = self._side(k, x)
            if k_new:
                out_k = self._new(k, stream)
            o = self._side(out_k, k)
            if out_k.shape != k.shape:
                raise ValueError("an output must have its input's shape")
            a.n_kv_heads, a.k, a.k_out = k.shape[1], k.data_ptr(), out_k.data_ptr()
            a.k_row_stride, a.k_head_stride, a.k_out_row_stride, a.k_out_head_stride = s[0], s[1], o[0], o[1]
        rc = self._lib.l2_rope(self._ref, ctypes.byref(a), self._raw_stream(index) if stream is None else stream.cuda_stream)
        if rc:
            _raise(rc)
        if stream is not None:  # their memory is kept until the call has run
            for t in (positions, q, k, None if q_new else out_q, None if k_new else out_k):
                if t is not None:
                    t.record_stream(stream)
        return out_q, out_k

    def _new(self, t, stream):
        torch = self._torch
        if stream is None:
            return torch.empty(t.shape, dtype=t.dtype, device=t.device)
        with torch.cuda.stream(stream):
            return torch.empty(t.shape, dtype=t.dtype, device=t.device)

    @staticmethod
    def _side(t, like):
        """Strides of q, k or an output, whose rows, head size, type and device are another's."""
        shape, want, st = t.shape, like.shape, t.stride()
        if len(shape) != 3 or shape[0] != want[0] or shape[2] != want[2] or t.dtype is not like.dtype or t.get_device() != like.get_device() \
                or (st[2] != 1 and shape[2] > 1):
            raise ValueError("q, k and outputs must be [rows][heads][head size] of one type and device, the last dimension contiguous")
        return st
