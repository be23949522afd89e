"""Slow and backward pairs at far positions on the GPU against 64 bits.

Tolerance as in tests/test_gpu_rope.py, (8.2 u) (|a| + |b|), u = 2^-24, and the angle's own error: |p| 2^-65 turns for the frequency as a fraction of a
turn, 2^-52 of p f for its quotient by 2 pi, and 2^-53 each for the product and the cosine's argument here.
"""
import math

import numpy as np
import pytest

from tests import tree_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402

U = 2.0 ** -24


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_slow_and_backward_pairs_at_far_positions(layout):
    freqs = [1e-12, -1e-12, 1e-9, -1e-9, -1e-7, 1e-16, 1e-20, -1.0, -0.01, 3e-8]
    rope = pkg.Rope(20, layout=layout, freqs=freqs)
    p = np.array([0, 1, -1, 8191, 10 ** 6, -10 ** 8, 2 ** 31 - 1, -2 ** 31], np.int64)
    x = torch.randn((len(p), 3, 24), device="cuda")
    out, _ = rope.apply(torch.tensor(p, dtype=torch.int32, device="cuda"), x)
    angle = p[:, None] * np.array(freqs)[None]
    x = x.double().cpu().numpy()
    want = tree_ref.rope(x, angle, 1.0, layout == "half")
    a, b = (slice(0, 10), slice(10, 20)) if layout == "half" else (slice(0, 20, 2), slice(1, 20, 2))
    off = 2 * math.pi * np.abs(p)[:, None] * 2.0 ** -65 + 2.0 ** -51 * np.abs(angle)
    size = (np.abs(x[..., a]) + np.abs(x[..., b])) * (8.2 * U + off[:, None])
    tol = np.zeros(x.shape)
    tol[..., a] = tol[..., b] = size
    tol += U * (np.abs(want) + tol)
    tol[..., 20:] = 0
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err - tol).max())


def test_backward_is_the_inverse_of_forward():
    """The same frequencies of the other sign at a position turn as these do at minus the position, bit for bit."""
    freqs = [1.0, 0.3, 1e-4, 1e-7, 1e-11, 12.5]
    there, back = pkg.Rope(12, freqs=freqs), pkg.Rope(12, freqs=[-f for f in freqs])
    x = torch.randn((40, 2, 12), device="cuda")
    p = torch.randint(-2 ** 31 + 1, 2 ** 31 - 1, (40,), dtype=torch.int64, device="cuda").int()
    assert torch.equal(there.apply(p, x)[0], back.apply(-p, x)[0])
