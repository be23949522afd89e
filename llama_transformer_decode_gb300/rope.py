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
        self._raw_stream = torch._C._cuda_getCurrentRawStream
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
        torch = self._torch
        x = q if q is not None else k
        if x is None or (q is None and out_q is not None) or (k is None and out_k is not None):
            raise ValueError("q, k or both, and an output only for one that is given")
        dtype, index = x.dtype, x.get_device()
        if dtype not in self._kinds or index < 0:
            raise ValueError("expected float32, bfloat16 or float16 CUDA tensors")
        rows, hs = x.shape[0], x.shape[-1]
        if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32 or positions.get_device() != index \
                or positions.dim() != 1 or positions.numel() != rows or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 tensor [{rows}] on the device of q and k")

        def side(t, out):
            if t is None:
                return None, (0, None, None, 0, 0, 0, 0), True
            self._check(t, dtype, index, rows, hs)
            fresh = out is None
            if fresh:
                if stream is None:
                    out = torch.empty(t.shape, dtype=dtype, device=t.device)
                else:
                    with torch.cuda.stream(stream):
                        out = torch.empty(t.shape, dtype=dtype, device=t.device)
            else:
                self._check(out, dtype, index, rows, hs)
                if out.shape != t.shape:
                    raise ValueError("an output must have its input's shape")
            a, b = t.stride(), out.stride()
            return out, (t.shape[1], t.data_ptr(), out.data_ptr(), a[0], a[1], b[0], b[1]), fresh

        q_out, (qh, qp, qo, qr, qs, qor, qos), q_new = side(q, out_q)
        k_out, (kh, kp, ko, kr, ks, kor, kos), k_new = side(k, out_k)
        a = L2RopeRows(rows, self._kinds[dtype], hs, qh, kh, positions.data_ptr(), qp, kp, qo, ko, qr, qs, kr, ks, qor, qos, kor, kos)
        rc = self._lib.l2_rope(self._ref, ctypes.byref(a), self._raw_stream(index) if stream is None else stream.cuda_stream)
        if rc:
            _raise(rc)
        if stream is not None:  # their memory is kept until the call has run
            for t in (positions, q, k, None if q_new else q_out, None if k_new else k_out):
                if t is not None:
                    t.record_stream(stream)
        return q_out, k_out

    @staticmethod
    def _check(t, dtype, index, rows, hs):
        if t.dim() != 3 or t.dtype is not dtype or t.get_device() != index or t.shape[0] != rows or t.shape[2] != hs \
                or (hs > 1 and t.stride(2) != 1):
            raise ValueError("q, k and outputs must be [rows][heads][head size] of one type and device, the last dimension contiguous")
