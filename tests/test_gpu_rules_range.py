"""Rules on logits over the whole range of their arguments, and before the sampler."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402
from tests.test_gpu_rules import DT, Made, check, dev, f32  # noqa: E402

U = 2.0 ** -24


@pytest.mark.parametrize("V", [64, 67])
def test_quotients_at_any_repetition_penalty(V):
    """l > 0 seen: l times the rounded inverse, two roundings of at most U of the quotient each (and half of the least subnormal); l <= 0: one."""
    rep = np.array([2.0 ** -126, 2.0 ** -100, 1e-20, 0.3, 0.7, 1.1, 3.0, 7e5, 2.0 ** 100, 1.9 * 2.0 ** 125, 2.0 ** 126], np.float32)
    n = len(rep)
    rules = pkg.TokenRules(V, dev(np.tile(np.arange(V), (n, 1))), dev([V] * n), repetition=f32(rep))
    rng = np.random.default_rng(V)
    x = (rng.uniform(0.13, 1.99, (n, V)) * rng.choice([-1, 1], (n, V))).astype(np.float32)
    got = rules.apply(torch.from_numpy(x).cuda())
    rules.check()
    r = rep.astype(np.float64)[:, None]
    want = np.where(x > 0, x / r, x * r)
    tol = np.where(x > 0, 2.001, 1) * U * np.abs(want) + 2.0 ** -150
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("bias", [0, 6])
@pytest.mark.parametrize("V,sizes", [(2048, [40] * 30), (16384, [64] * 9), (8192 + 8, [33] * 20), (8192 + 4, [33] * 20)])
def test_trees_of_every_kernel(V, sizes, bias, dtype, out):
    """Rows that come in trees, several to a block, with biases and without, 16 and 8 bytes an access."""
    n = len(sizes)
    m = Made(V, n, 50, V + n, bias=bias)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    rows = int(starts[-1])
    drafted = m.rng.integers(0, 40, rows)
    parents = np.concatenate([[-1] + [int(m.rng.integers(0, u)) for u in range(1, k)] for k in sizes])
    logits = (torch.randn((rows, V), device="cuda") * 3).to(DT[dtype])
    which = m.rng.integers(-1, 5, rows)
    got = m.rules.apply(logits, starts=dev(starts), parents=dev(parents), drafted=dev(drafted), masks=m.packed(), mask_rows=dev(which), out_dtype=DT[out])
    m.rules.check()
    x = logits.double().cpu().numpy()
    for i in range(n):
        for u in sorted({0, sizes[i] - 1, *m.rng.integers(0, sizes[i], 4).tolist()}):
            r, path, at = int(starts[i]) + u, [], u
            while at >= 0:
                path.append(int(drafted[starts[i] + at]))
                at = int(parents[starts[i] + at])
            check(got[r], *m.row(x[r], i, path, None if which[r] < 0 else int(which[r])))
    again = logits.clone()
    if out == dtype:
        m.rules.apply(again, starts=dev(starts), parents=dev(parents), drafted=dev(drafted), masks=m.packed(), mask_rows=dev(which), out=again)
        assert torch.equal(again.view(torch.uint8), got.view(torch.uint8))


def test_the_samplers_vocabulary_is_smaller_than_the_rules():
    """Rules take up to 2^24 tokens, the sampler 49152: more than that it refuses before anything runs."""
    for V, fits in ((49152, True), (49153, False), (128000, False)):
        rules = pkg.TokenRules(V, dev(np.zeros((2, 1))), dev([0, 0]))
        masks = torch.zeros((2, -(-V // 32)), dtype=torch.int32, device="cuda")
        masks[1, V // 64] = 1
        logits = rules.apply(torch.randn((2, V), device="cuda"), masks=masks)
        rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
        tokens = torch.full((2,), -5, dtype=torch.int32, device="cuda")
        if fits:
            pkg.sample(logits, 0.8, 0.9, rng, out=tokens)
            assert tokens.tolist() == [0, V // 64 * 32]
        else:
            with pytest.raises(pkg.L2Error, match="49152"):
                pkg.sample(logits, 0.8, 0.9, rng, out=tokens)
            assert tokens.tolist() == [-5, -5] and rng.tolist() == [5, 6]
            assert bool((logits[0] == -float("inf")).all()) and int(logits[1].argmax()) == V // 64 * 32
