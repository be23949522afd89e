"""Rotary positions on the GPU against 64 bits.

Tolerance, element by element (u = 2^-24): the angle within half a turn is rounded to fp32 (off by at most pi u), cosine and sine
are within one unit in the last place (2 u) and are multiplied by the amplitude (u), so each is off by at most 6.2 u; the frequency as a
fraction of 2^64 adds 3 * 2^-53 of the whole angle; two products and a sum add 2 u: (8.2 u + 4 * 2^-53 |p f|) (|a| + |b|) amplitude, and half a
step of the type for the result.
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

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24


def check(got, x, positions, rope, amplitude=1.0):
    dtype = x.dtype
    pos = positions.cpu().numpy().astype(np.float64)
    angle = pos[:, None] * np.array(rope.freqs)[None]
    half = rope.layout == "half"
    x = x.double().cpu().numpy()
    want = tree_ref.rope(x, angle, amplitude, half)
    rot = rope.rot_dim
    size = np.zeros(x.shape)
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if half else (slice(0, rot, 2), slice(1, rot, 2))
    both = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(amplitude) * (8.2 * U + 4 * 2.0 ** -53 * np.abs(angle)[:, None])
    size[..., a] = size[..., b] = both
    step = torch.finfo(dtype).eps / 2
    tol = size + step * (np.abs(want) + size) + (2.0 ** -25 if dtype is torch.float16 else 1e-45)
    tol[..., rot:] = 0          # what does not turn stays as it is
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err - tol).max())


def positions_of(n, far, seed=0, negative=False):
    p = np.random.default_rng(seed).integers(-far if negative else 0, far + 1, n)
    p[:1] = far
    return torch.tensor(p, dtype=torch.int32, device="cuda")


CASES = [
    # query heads, kv heads, head size, rot_dim, rows, farthest position
    (32, 8, 128, 128, 64, 8192),
    (8, 4, 8, 8, 1, 100),
    (6, 4, 48, 48, 17, 1000),
    (12, 12, 64, 32, 130, 100000),     # half of the head
    (3, 1, 24, 10, 5, 50),             # 5 pairs: single elements
    (5, 2, 20, 4, 33, 2 ** 31 - 1),
    (2, 2, 256, 256, 7, 1000000),      # the largest head
    (1, 1, 2, 2, 3, 10),               # the smallest
    (4, 0, 64, 64, 9, 5000),           # queries alone
    (0, 4, 64, 64, 9, 5000),           # keys alone
    (64, 8, 128, 64, 3000, 1000000),   # many rows
    (1, 1, 7, 6, 400, 20),             # odd head size
    (40, 1, 100, 24, 2, 300),
]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_rotations_match_64_bits(case, dtype, layout):
    H, KV, hs, rot, rows, far = CASES[case]
    rope = pkg.Rope(rot, layout=layout)
    g = torch.Generator(device="cuda").manual_seed(case)
    wide = torch.randn((rows, H + 2 * KV + 1, hs), generator=g, device="cuda").to(DT[dtype])   # a fused projection
    q, k = wide[:, :H] if H else None, wide[:, H:H + KV] if KV else None
    pos = positions_of(rows, far, case, negative=case % 2 == 1)
    before = wide.clone()
    oq, ok = rope.apply(pos, q, k)
    assert torch.equal(wide, before)
    for got, x in ((oq, q), (ok, k)):
        assert (got is None) == (x is None)
        if x is not None:
            check(got, x, pos, rope)
    # in place, within the projection: the same bits, and nothing else changes
    rope.apply(pos, q, k, out_q=q, out_k=k)
    if H:
        assert torch.equal(wide[:, :H], oq)
    if KV:
        assert torch.equal(wide[:, H:H + KV], ok)
    assert torch.equal(wide[:, H + KV:], before[:, H + KV:])
    # heads outside rows, into other columns of one matrix
    if H and KV:
        t = before[:, :H].transpose(0, 1).contiguous().transpose(0, 1)
        room = torch.full((rows, H + KV + 3, hs), 3.0, device="cuda").to(DT[dtype])
        rope.apply(pos, t, before[:, H:H + KV], out_q=room[:, 1:H + 1], out_k=room[:, H + 1:H + 1 + KV])
        assert torch.equal(room[:, 1:H + 1], oq) and torch.equal(room[:, H + 1:H + 1 + KV], ok)
        assert bool((room[:, 0] == 3.0).all()) and bool((room[:, H + 1 + KV:] == 3.0).all())


@pytest.mark.parametrize("offset", [1, 2, 4, 8])
def test_addresses_at_any_element(offset):
    rope = pkg.Rope(32, layout="half")
    for dtype in DT.values():
        flat = torch.randn(6 * 5 * 40 + offset, device="cuda").to(dtype)
        x = flat[offset:].view(6, 5, 40)
        pos = positions_of(6, 1000)
        out, _ = rope.apply(pos, x)
        check(out, x, pos, rope)


@pytest.mark.parametrize("kind", [dict(kind="linear", factor=4.0), dict(kind="base", factor=8.0), dict(kind="linear", factor=0.5),
                                  dict(kind="bands", factor=8.0, original_len=8192.0, low=1.0, high=4.0, amplitude=1.25),
                                  dict(freqs=[1.0, -0.5, 0.0, 7.5, 1e-9, 100.0, 0.25, 3.0])])
def test_scaled_and_own_frequencies(kind):
    rot = 16
    rope = pkg.Rope(rot, base=500000.0, **kind)
    f = 500000.0 ** (-np.arange(0, rot, 2) / rot)
    if "freqs" in kind:
        f = np.array(kind["freqs"])
    elif kind["kind"] == "linear":
        f = f / kind["factor"]
    elif kind["kind"] == "base":
        f = (500000.0 * 8.0 ** (16 / 14)) ** (-np.arange(0, rot, 2) / rot)
        assert math.isclose(f[-1], 500000.0 ** (-14 / 16) / 8.0, rel_tol=1e-12) and f[0] == 1.0
    else:
        s = np.clip((8192.0 * f / (2 * math.pi) - 1.0) / 3.0, 0, 1)
        f = f * (s + (1 - s) / 8.0)
        assert 0 < s[2] or s[0] == 1
    assert np.allclose(rope.freqs, f, rtol=1e-12, atol=0)
    x = torch.randn((50, 3, 24), device="cuda")
    pos = positions_of(50, 200000, negative=True)
    out, _ = rope.apply(pos, x)
    check(out, x, pos, rope, kind.get("amplitude", 1.0))


def test_the_decoders_own_rotation():
    """Base 10000, neighbours as pairs: the keys that the decoder's step leaves in its cache."""
    import synth
    wl = synth.WORKLOADS["tiny"]
    w = synth.make_weights(wl)
    dec = pkg.Decoder(wl.config_tuple(), pkg.to_device(w))
    toks = synth.token_stream(wl, 0, 6)
    for pos, tok in enumerate(toks):
        dec.forward(int(tok), pos)
    k, _ = dec.kv_export(0)
    emb = np.stack([w["emb"][int(t)] for t in toks]).astype(np.float64)
    x = emb / np.sqrt((emb ** 2).mean(axis=1, keepdims=True) + 1e-5) * w["rms_att"][0]
    keys = torch.tensor((x @ w["wk"][0].reshape(-1, wl.dim).T.astype(np.float64)).astype(np.float32), device="cuda").view(len(toks), wl.n_kv_heads, wl.head_size)
    rope = pkg.Rope(wl.head_size)
    _, out = rope.apply(torch.arange(len(toks), dtype=torch.int32, device="cuda"), k=keys)
    got = out.reshape(len(toks), -1).cpu().numpy()
    # both are fp32 sums of dim products, in other orders
    size = np.abs(x) @ np.abs(w["wk"][0].reshape(-1, wl.dim).T)
    tol = (size.reshape(len(toks), -1, 2).sum(axis=2, keepdims=True) * (wl.dim + 40) * 2 * U).repeat(2, axis=2).reshape(got.shape)
    assert (np.abs(got - k) <= tol).all()
    dec.close()


def test_a_shift_is_a_rotation_by_the_difference():
    """Keys in a cache move to other positions by turning them again, to a negative one as well."""
    rope = pkg.Rope(64, layout="half")
    x = torch.randn((40, 2, 64), device="cuda")
    a, b = positions_of(40, 5000, 1), positions_of(40, 5000, 2)
    _, at_a = rope.apply(a, k=x)
    _, at_b = rope.apply(b, k=x)
    _, moved = rope.apply(b - a, k=at_a)
    size = x.abs()[..., :32] + x.abs()[..., 32:]
    tol = (3 * 8.2 + 6) * U * torch.cat([size, size], dim=-1) * 1.5
    assert bool(((moved - at_b).abs() <= tol).all())


def test_empty_calls_graphs_and_streams():
    rope = pkg.Rope(64)
    none, _ = rope.apply(torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty((0, 4, 64), device="cuda"))
    assert none.shape == (0, 4, 64)
    x = torch.randn((16, 4, 64), device="cuda").to(torch.bfloat16)
    pos = positions_of(16, 100)
    out = torch.empty_like(x)
    rope.apply(pos, x, out_q=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.apply(pos, x, out_q=out)
    for seed in range(3):
        x.normal_()
        pos.copy_(positions_of(16, 10 ** 6, seed))
        graph.replay()
        check(out, x, pos, rope)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        y, p2 = x.clone(), pos.clone()
    got, _ = rope.apply(p2, y, stream=st)
    del y, p2
    torch.empty(16 * 4 * 64, dtype=torch.bfloat16, device="cuda").fill_(9)
    torch.cuda.synchronize()
    assert torch.equal(got, out)


def test_rotations_the_host_refuses():
    rope = pkg.Rope(32)
    pos = positions_of(8, 10)
    x = torch.randn((8, 4, 64), device="cuda")
    with pytest.raises(ValueError):
        rope.apply(pos)
    with pytest.raises(ValueError):
        rope.apply(pos[:7], x)
    with pytest.raises(ValueError):
        rope.apply(pos.long(), x)
    with pytest.raises(ValueError):
        rope.apply(pos, x.double())
    with pytest.raises(ValueError):
        rope.apply(pos, x, x.to(torch.bfloat16))
    with pytest.raises(ValueError):
        rope.apply(pos, x, out_k=x)
    with pytest.raises(ValueError):
        rope.apply(pos, x, out_q=torch.empty((8, 3, 64), device="cuda"))
    with pytest.raises(ValueError):
        rope.apply(pos, x.transpose(1, 2))
    with pytest.raises(pkg.L2Error, match="head_size"):
        rope.apply(pos, x[..., :16])
    with pytest.raises(pkg.L2Error, match="overlap"):
        rope.apply(pos, x, out_q=torch.empty((1, 4, 64), device="cuda").expand(8, 4, 64))
    flat = torch.zeros(9 * 4 * 64, device="cuda")
    with pytest.raises(pkg.L2Error, match="shares memory"):
        rope.apply(pos, flat[:8 * 256].view(8, 4, 64), out_q=flat[256:].view(8, 4, 64))
    with pytest.raises(pkg.L2Error, match="shares memory"):
        rope.apply(pos, x, x, out_q=x, out_k=torch.empty_like(x))
    wide = torch.zeros((8, 6, 64), device="cuda")
    with pytest.raises(pkg.L2Error, match="shares memory"):
        rope.apply(pos, x, x, out_q=wide[:, :4], out_k=wide[:, 2:])
    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=258), dict(rot_dim=8, base=0.0), dict(rot_dim=8, base=math.inf),
                dict(rot_dim=8, kind="linear", factor=0.0), dict(rot_dim=8, kind="bands", factor=2.0, original_len=0.0),
                dict(rot_dim=8, kind="bands", factor=2.0, original_len=9.0, low=4.0, high=4.0), dict(rot_dim=8, amplitude=math.nan),
                dict(rot_dim=4, freqs=[1.0, math.nan])):
        with pytest.raises(pkg.L2Error):
            pkg.Rope(**bad)
    for bad in (dict(rot_dim=8, layout="other"), dict(rot_dim=8, kind="other"), dict(rot_dim=8, freqs=[1.0])):
        with pytest.raises(ValueError):
            pkg.Rope(**bad)
