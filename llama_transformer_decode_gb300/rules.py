"""Rules on logits before sampling: penalties for tokens that a sequence already holds, biases, grammar
masks (``l2_token_rules`` of ``include/l2.h``).  ``sample`` draws from what they leave, where the vocabulary has at most
49152 tokens; rules take up to 2^24.

Arguments are marshalled here; counting and arithmetic are the CUDA kernel's.  Calls enqueue on
``stream`` (default: torch's current stream), never wait, and can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes

from . import _native
from ._native import L2TokenRows, L2TokenRules

_L2_EDEVICE = -5


def _raise(code: int):
    from . import L2Error
    raise L2Error(code, _native.load().l2_last_error(None).decode())


class TokenRules:
    """The rules of ``n_seqs`` sequences over a vocabulary of ``vocab_size`` tokens.

    ``history`` [n_seqs][room] and ``lens`` [n_seqs]: int32 CUDA tensors, the tokens each sequence holds; the caller changes them as
    sequences grow.  ``repetition``, ``presence``, ``frequency``: float32 [n_seqs] or None (``repetition`` above 0).  ``counted_from``: int32 [n_seqs] or
    None, where the latter two begin to count.  ``bias``: (starts int32 [n_seqs + 1], tokens int32, values float32) or None: entries
    starts[s]..starts[s + 1] - 1 are sequence s's.  All are kept, and read by each call when it runs.
    """

    def __init__(self, vocab_size: int, history, lens, counted_from=None, repetition=None, presence=None, frequency=None, bias=None):
        import torch
        self._torch, self._lib = torch, _native.load()
        self._raw_stream, self._int32 = torch._C._cuda_getCurrentRawStream, torch.int32
        self._kinds = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        if not isinstance(history, torch.Tensor) or history.dim() != 2 or history.dtype is not torch.int32 or not history.is_cuda \
                or (history.shape[1] > 1 and history.stride(1) != 1):
            raise ValueError("history must be an int32 CUDA tensor [sequences][room], its last dimension contiguous")
        self.device, self._index, self.vocab_size = history.device, history.get_device(), int(vocab_size)
        n = self.n_seqs = history.shape[0]
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

        def one(name, t, dtype, count):
            if t is None:
                return None
            if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != self._index or t.dim() != 1 or not t.is_contiguous() \
                    or (count is not None and t.numel() != count):
                raise ValueError(f"{name} must be a contiguous {dtype} tensor [{'n' if count is None else count}] on {self.device}")
            return t.data_ptr()

        if lens is None:
            raise ValueError("lens is needed")
        b = (None, None, None) if bias is None else tuple(bias)
        if len(b) != 3 or (bias is not None and (any(t is None for t in b) or len(b[1]) != len(b[2]))):
            raise ValueError("bias must be (starts, tokens, values), with as many tokens as values")
        self._kept = (history, lens, counted_from, repetition, presence, frequency, *b)
        self._c = L2TokenRules(n, self.vocab_size, history.shape[1], 0 if bias is None else len(b[1]), history.stride(0), history.data_ptr(),
                               one("lens", lens, torch.int32, n), one("counted_from", counted_from, torch.int32, n),
                               one("repetition", repetition, torch.float32, n), one("presence", presence, torch.float32, n),
                               one("frequency", frequency, torch.float32, n), one("bias starts", b[0], torch.int32, n + 1),
                               one("bias tokens", b[1], torch.int32, None), one("bias values", b[2], torch.float32, None), self.status.data_ptr())
        self._ref = ctypes.byref(self._c)
        rc = self._lib.l2_token_rules_init(self._ref)
        if rc:
            _raise(rc)

    def _ints(self, name, t, n=None):
        """Address of an index array; n: its length, where the call fixes it."""
        if not isinstance(t, self._torch.Tensor) or t.dtype is not self._int32 or t.get_device() != self._index or t.dim() != 1 \
                or not t.is_contiguous() or (n is not None and t.numel() != n):
            raise ValueError(f"{name} must be a contiguous int32 tensor [{'n' if n is None else n}] on {self.device}")
        return t.data_ptr()

    def _matrix(self, name, t):
        """Rows and row stride of logits."""
        shape, st = t.shape, t.stride()
        if len(shape) != 2 or shape[1] != self.vocab_size or t.dtype not in self._kinds or t.get_device() != self._index \
                or (st[1] != 1 and shape[1] > 1):
            raise ValueError(f"{name} must be [rows][{self.vocab_size}], float32, bfloat16 or float16 on {self.device}, its last dimension contiguous")
        return shape[0], st[0]

    def _new(self, rows, dtype, stream):
        torch = self._torch
        if stream is None:
            return torch.empty((rows, self.vocab_size), dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty((rows, self.vocab_size), dtype=dtype, device=self.device)

    def check(self):
        """Waits for the device and raises L2Error if a row could not be done (and clears the status)."""
        self._torch.cuda.synchronize(self.device)
        if int(self.status.item()):
            from . import L2Error
            self.status.zero_()
            raise L2Error(_L2_EDEVICE, "token rules: rows with an invalid sequence, tree, length or mask number")

    def apply(self, logits, seqs=None, starts=None, parents=None, drafted=None, masks=None, mask_rows=None, out=None, out_dtype=None,
              stream=None):
        """The rules applied to ``logits`` ([rows][vocab_size], float32, bfloat16 or float16).

        Row i is of sequence seqs[i] (i, without ``seqs``), or with ``starts`` rows starts[i]..starts[i + 1] - 1 are, the tokens of a
        tree: ``drafted`` are the rows' own tokens and ``parents`` their trees as for ``PagePool.tree_attention``, and a row is
        penalised for its path, too.  ``masks`` (int32 [masks][ceil(vocab_size / 32)], bit v % 32 of word v / 32 set where token v is
        allowed): row r's is masks[mask_rows[r]] (-1: none), or masks[r].  Returns ``out`` (in place: ``logits``), by default a
        new tensor of ``out_dtype`` (float32 or the logits' type, which is the default; ``sample`` takes float32)."""
        kinds, ints, V = self._kinds, self._ints, self.vocab_size
        rows, row_stride = self._matrix("logits", logits)
        n = rows if starts is None else starts.shape[0] - 1
        if parents is not None and starts is None:
            raise ValueError("parents need starts")
        fresh = out is None
        if fresh:
            dtype = logits.dtype if out_dtype is None else out_dtype
            if dtype not in kinds:
                raise ValueError("out_dtype must be float32 or the logits' type")
            out, out_stride = self._new(rows, dtype, stream), V
        else:
            dtype = out.dtype
            out_rows, out_stride = self._matrix("out", out)
            if out_rows != rows or (out_dtype is not None and dtype is not out_dtype):
                raise ValueError("out must have the logits' rows, and out_dtype's type")
        a = L2TokenRows(n, rows, None if seqs is None else ints("seqs", seqs, n), None if starts is None else ints("starts", starts),
                        None if parents is None else ints("parents", parents, rows), None if drafted is None else ints("drafted", drafted, rows),
                        logits.data_ptr(), out.data_ptr(), kinds[logits.dtype], kinds[dtype], row_stride, out_stride)
        if masks is not None:
            shape, words = masks.shape, -(-V // 32)
            if masks.dtype is not self._int32 or len(shape) != 2 or masks.get_device() != self._index or shape[1] != words \
                    or (words > 1 and masks.stride(1) != 1):
                raise ValueError(f"masks must be int32 [masks][{words}] on {self.device}, the last dimension contiguous")
            a.masks, a.mask_stride, a.n_masks = masks.data_ptr(), masks.stride(0), shape[0]
            if mask_rows is not None:
                a.mask_rows = ints("mask_rows", mask_rows, rows)
        elif mask_rows is not None:
            raise ValueError("mask_rows needs masks")
        if rows == 0:
            return out
        rc = self._lib.l2_token_rules(self._ref, ctypes.byref(a), self._raw_stream(self._index) if stream is None else stream.cuda_stream)
        if rc:
            _raise(rc)
        if stream is not None:  # their memory is kept until the call has run
            for t in (logits, seqs, starts, parents, drafted, masks, mask_rows, None if fresh else out, *self._kept, self.status):
                if t is not None:
                    t.record_stream(stream)
        return out
