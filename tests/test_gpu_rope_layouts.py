"""Rotary positions where queries, keys and outputs lie in one piece of memory: everything that shares no byte is turned, everything that shares
one is refused (in place apart)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402
from tests.test_gpu_rope import DT, check, positions_of  # noqa: E402


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,H,kv,hs,rot,order", [
    (9, 8, 8, 64, 32, "heads then parts"),      # [rows][heads][q, k, v][head size]: models with half pairs and partial rotation
    (1, 16, 16, 128, 128, "heads then parts"),
    (300, 4, 2, 24, 10, "heads then parts"),    # the first heads alone have keys
    (5, 1, 1, 64, 64, "heads then parts"),
    (17, 6, 6, 48, 48, "heads outside"),        # [heads][rows][q, k, v][head size]
    (17, 6, 1, 48, 48, "parts between"),        # [heads][q, k, v][rows][head size]
    (12, 3, 3, 7, 6, "heads then parts"),
])
def test_parts_of_each_head_side_by_side(rows, H, kv, hs, rot, order, dtype, layout):
    g = torch.Generator(device="cuda").manual_seed(rows)
    shape, dims = {"heads then parts": ((rows, H, 3, hs), (0, 1, 2, 3)), "heads outside": ((H, rows, 3, hs), (1, 0, 2, 3)),
                   "parts between": ((H, 3, rows, hs), (2, 0, 1, 3))}[order]
    fused = torch.randn(shape, generator=g, device="cuda").to(DT[dtype]).permute(dims)      # [rows][heads][part][head size]
    q, k = fused[:, :, 0], fused[:, :kv, 1]
    before = fused.clone()
    rope = pkg.Rope(rot, layout=layout)
    pos = positions_of(rows, 3000, rows)
    oq, ok = rope.apply(pos, before[:, :, 0], before[:, :kv, 1])
    check(oq, before[:, :, 0], pos, rope)
    check(ok, before[:, :kv, 1], pos, rope)
    rope.apply(pos, q, k, out_q=q, out_k=k)                 # in place, both in one call
    assert torch.equal(q, oq) and torch.equal(k, ok)
    rest = fused.clone()
    rest[:, :, 0], rest[:, :kv, 1] = before[:, :, 0], before[:, :kv, 1]
    assert torch.equal(rest, before)                        # values, and keys of the other heads
    # from one part to another one
    v = fused[:, :kv, 2]
    rope.apply(pos, None, before[:, :kv, 1], out_k=v)
    assert torch.equal(v, ok)
    if H == kv:
        fused.copy_(before)
        rope.apply(pos, fused[:, :, 0], out_q=fused[:, :, 2])
        assert torch.equal(fused[:, :, 2], oq) and torch.equal(fused[:, :, :2], before[:, :, :2])


@pytest.mark.parametrize("seed", range(4))
def test_exactly_what_shares_memory_is_refused(seed):
    """Queries and keys at random places of one buffer, with the rows' strides alike, against sets of elements."""
    rng = np.random.default_rng(seed)
    rope = pkg.Rope(4)
    flat = torch.randn(6000, device="cuda")
    seen = {True: 0, False: 0}
    for turn in range(250):
        rows, hs, H, kv = int(rng.integers(1, 6)), int(rng.integers(4, 9)), int(rng.integers(1, 5)), int(rng.integers(1, 5))
        head = int(rng.integers(hs, 4 * hs))
        row = int(rng.integers(hs, 6 * hs * max(H, kv)))
        other = head if turn % 2 else int(rng.integers(hs, 4 * hs))
        a = int(rng.integers(0, 400))
        b = a + int(rng.integers(-min(a, 200), 200))
        of = lambda at, n, h: [at + r * row + i * h + e for r in range(rows) for i in range(n) for e in range(hs)]  # noqa: E731
        left, right = of(a, H, head), of(b, kv, other)
        if len(set(left)) < len(left) or len(set(right)) < len(right) or max(left + right) >= 6000:
            continue
        ordered = lambda n, h: n == 1 or rows == 1 or row >= (n - 1) * h + hs or h >= (rows - 1) * row + hs  # noqa: E731
        if not ordered(H, head) or not ordered(kv, other):  # rows that are woven into heads: refused for themselves
            continue
        share = bool(set(left) & set(right))
        seen[share] += 1
        q, k = flat.as_strided((rows, H, hs), (row, head, 1), a), flat.as_strided((rows, kv, hs), (row, other, 1), b)
        pos = positions_of(rows, 1000, turn)
        before = flat.clone()
        if share:
            with pytest.raises(pkg.L2Error, match="shares memory"):
                rope.apply(pos, q, k, out_q=q, out_k=k)
            assert torch.equal(flat, before)
        else:
            oq, ok = rope.apply(pos, q, k)
            rope.apply(pos, q, k, out_q=q, out_k=k)
            assert torch.equal(q, oq) and torch.equal(k, ok)
            rest = torch.ones(6000, dtype=torch.bool, device="cuda")
            rest[torch.tensor(left + right, device="cuda")] = False
            assert torch.equal(flat[rest], before[rest])
    assert min(seen.values()) > 20


def test_far_rows_count_as_memory():
    """What meets is a late row of one and an early row of the other, or a late head."""
    rope = pkg.Rope(8)
    flat = torch.randn(20000, device="cuda")
    pos = positions_of(9, 10)
    view = lambda at, row, head, n=4: flat.as_strided((9, n, 8), (row, head, 1), at)  # noqa: E731
    q = view(0, 300, 24)
    for at in (8 * 300 + 3 * 24 + 7, 2100 + 5, 300 + 24 + 23):
        k = view(at, 300, 24)
        with pytest.raises(pkg.L2Error, match="shares memory"):
            rope.apply(pos, q, k, out_q=q, out_k=k)
    for at in (8, 16, 300 + 8, 8 * 300 + 3 * 24 + 8, 8 * 300 + 16):
        k = view(at, 300, 24)
        oq, ok = rope.apply(pos, q, k)
        rope.apply(pos, q, k, out_q=q, out_k=k)
        assert torch.equal(q, oq) and torch.equal(k, ok)
