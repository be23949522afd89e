"""Rules on logits on the GPU against the plain statement in 64 bits.

Tolerance (u = 2^-24, m = |l| max(r, 1 / r) + |frequency| n + |presence| + |bias|): a quotient, as a product with the rounded inverse, rounds twice,
frequency * n + presence once, their difference and the bias' sum once each, by at most u of what they round: 2 |l / r| + (|frequency| n +
|presence|) + 2 m is at most 4 m, so 4 u m, and half a step of a 16-bit result.
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


def dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def f32(a):
    return torch.tensor(np.asarray(a), dtype=torch.float32, device="cuda")


class Made:
    """Sequences with histories, penalties, biases and masks, on the host and on the GPU."""

    def __init__(self, V, n, room, seed, penalties=True, bias=6, masks=5):
        rng = self.rng = np.random.default_rng(seed)
        self.V, self.n = V, n
        self.lens = rng.integers(0, room + 1, n)
        self.lens[0] = room
        # some tokens often, some outside the vocabulary, as placeholders are
        self.history = np.minimum((V * rng.random((n, room)) ** 3).astype(int), V - 1)
        if room > 3:
            self.history[:, 1] = -1
            self.history[:, 2] = V
            self.history[:, 3] = 2 ** 31 - 1
        self.counted = rng.integers(0, room + 2, n)
        self.rep, self.pres, self.freq = rng.uniform(0.7, 1.6, n), rng.uniform(-1, 1, n), rng.uniform(-0.5, 0.8, n)
        if n > 1:
            self.rep[1], self.pres[1], self.freq[1] = 1, 0, 0     # a sequence without penalties
        self.rep, self.pres, self.freq = (x.astype(np.float32) for x in (self.rep, self.pres, self.freq))
        self.bias = [[(int(rng.integers(0, V)), np.float32(rng.normal(0, 3))) for _ in range(rng.integers(0, bias + 1))] for _ in range(n)]
        if bias:
            self.bias[0] += [(V - 1, np.float32(2)), (V, np.float32(9)), (-1, np.float32(9)), (V - 1, np.float32(-math.inf)), (0, np.float32(4)),
                             (0, np.float32(1.5))]                # outside the vocabulary; one token twice: the last entry counts
        self.masks = rng.random((masks, V)) < rng.random((masks, 1)) if masks else None
        if masks:
            self.masks[0] = False                                 # nothing is allowed
            self.masks[-1] = True
        self.penalties = penalties
        flat = [e for b in self.bias for e in b]
        self.rules = pkg.TokenRules(V, dev(self.history), dev(self.lens), counted_from=dev(self.counted) if penalties else None,
                                    repetition=f32(self.rep) if penalties else None, presence=f32(self.pres) if penalties else None,
                                    frequency=f32(self.freq) if penalties else None,
                                    bias=(dev(np.concatenate([[0], np.cumsum([len(b) for b in self.bias])])), dev([t for t, _ in flat]),
                                          f32([v for _, v in flat])) if bias else None)

    def packed(self):
        words = -(-self.V // 32)
        bits = np.zeros((len(self.masks), words * 32), np.uint8)
        bits[:, :self.V] = self.masks
        bits[:, self.V:] = 1
        return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).cuda()

    def row(self, logits, s, path, mask):
        r, a, f = (float(x[s]) if self.penalties else d for x, d in ((self.rep, 1.0), (self.pres, 0.0), (self.freq, 0.0)))
        h = self.history[s, :self.lens[s]]
        want = tree_ref.rules(logits, h, self.counted[s] if self.penalties else 0, path, r, a, f, self.bias[s], None if mask is None else self.masks[mask])
        n = np.bincount([t for t in list(h) + list(path) if 0 <= t < self.V], minlength=self.V)
        b = np.zeros(self.V)
        for t, v in dict(self.bias[s]).items():
            if 0 <= t < self.V and np.isfinite(v):
                b[t] = abs(v)
        return want, np.abs(logits) * max(r, 1 / r) + abs(f) * n + abs(a) + b


def check(got, want, size):
    half = torch.finfo(got.dtype).eps / 2
    got = got.double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    tol = 4 * U * size + (half * (np.abs(np.where(fine, want, 0)) + 4 * U * size) + 2.0 ** -25 if half > U else 0)
    err = np.abs(np.where(fine, got - np.where(fine, want, 0), 0))
    assert (err <= np.where(fine, tol, 1)).all(), float((err - np.where(fine, tol, 1)).max())


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,n,room", [(1, 1, 4), (5, 2, 9), (512, 3, 40), (1023, 4, 200), (1025, 3, 0), (8193, 2, 3000), (32000, 5, 700), (50000, 64, 50)])
def test_rows_of_a_batch(V, n, room, dtype):
    m = Made(V, n, room, V + n)
    order = m.rng.integers(0, n, n + 2)                           # a sequence may come twice
    wide = torch.randn((n + 2, V + 3), device="cuda").mul(3).to(DT[dtype])
    for logits in (wide[:, :V], wide[:, :V].contiguous(), wide[:, 3:]):   # rows at odd addresses, and at even ones
        which = m.rng.integers(-1, 5, n + 2)
        which[0] = 0
        out = m.rules.apply(logits, seqs=dev(order), masks=m.packed(), mask_rows=dev(which), out_dtype=torch.float32)
        same = m.rules.apply(logits, seqs=dev(order), masks=m.packed(), mask_rows=dev(which))
        m.rules.check()
        assert out.dtype is torch.float32 and same.dtype is DT[dtype]
        x = logits.double().cpu().numpy()
        for r in range(n + 2):
            want, size = m.row(x[r], int(order[r]), [], None if which[r] < 0 else int(which[r]))
            check(out[r], want, size)
            check(same[r], want, size)
        # in place: the same bits
        before, rest = logits.clone(), wide.clone()
        m.rules.apply(logits, seqs=dev(order), masks=m.packed(), mask_rows=dev(which), out=logits)
        assert torch.equal(logits.contiguous().view(torch.uint8), same.view(torch.uint8))
        logits.copy_(before)
        assert torch.equal(wide, rest)


@pytest.mark.parametrize("parts", [dict(penalties=False), dict(bias=0), dict(masks=0), dict(penalties=False, bias=0, masks=0), dict(bias=0, masks=0)])
def test_some_rules_alone(parts):
    m = Made(777, 4, 30, 5, **parts)
    logits = torch.randn((4, 777), device="cuda") * 3
    masks = m.packed()[:4] if m.masks is not None else None      # without mask_rows: row r has mask r
    out = m.rules.apply(logits, masks=masks)
    m.rules.check()
    for r in range(4):
        want, size = m.row(logits[r].double().cpu().numpy(), r, [], r if masks is not None else None)
        check(out[r], want, size)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,sizes,kind", [(600, [7], "wide"), (32000, [5, 0, 64, 1, 33], "wide"), (128000, [20] * 6, "wide"), (3001, [3] * 40, "chain"),
                                          (40, [64, 64], "deep")])
def test_rows_of_trees_count_their_own_path(V, sizes, kind, dtype):
    n = len(sizes)
    m = Made(V, n, 60, n * 7 + V)
    trees = [tree_ref.chain(k) if kind == "chain" else tree_ref.random_tree(m.rng, k, back=3 if kind == "deep" else None) for k in sizes]
    order = m.rng.permutation(n)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    rows = int(starts[-1])
    drafted = np.minimum((V * m.rng.random(rows) ** 3).astype(int), V - 1)
    drafted[::5] = np.where(m.rng.random(len(drafted[::5])) < 0.3, -7, drafted[::5])
    logits = (torch.randn((rows + 2, V), device="cuda") * 3).to(DT[dtype])
    which = m.rng.integers(-1, 5, rows + 2)
    out = torch.full((rows + 2, V), 5.0, device="cuda")
    par = None if kind == "chain" else dev(list(np.concatenate([np.array(t, int) for t in trees])) + [9, 9])
    args = dict(seqs=dev(order), starts=dev(starts), parents=par, masks=m.packed(), mask_rows=dev(which))
    m.rules.apply(logits, drafted=dev(list(drafted) + [0, 0]), out=out, **args)
    m.rules.check()
    assert bool((out[rows:] == 5.0).all())                        # rows behind the last tree
    plain = m.rules.apply(logits, out=out.clone(), **args)        # without drafted: no path counts
    x = logits.double().cpu().numpy()
    for i in range(n):
        for u in range(sizes[i]):
            r = int(starts[i]) + u
            mask = None if which[r] < 0 else int(which[r])
            path = [int(drafted[starts[i] + j]) for j in tree_ref.line(trees[i], u)]
            check(out[r], *m.row(x[r], int(order[i]), path, mask))
            check(plain[r], *m.row(x[r], int(order[i]), [], mask))


def test_infinite_and_nan_logits():
    rules = pkg.TokenRules(6, dev([[0, 1, 2, 3]]), dev([4]), repetition=f32([2.0]), presence=f32([1.0]))
    x = f32([[math.inf, -math.inf, math.nan, 2.0, math.nan, math.inf]])
    out = rules.apply(x)
    assert out.cpu().tolist()[0][:2] == [math.inf, -math.inf] and bool(out[0, 2].isnan()) and float(out[0, 3]) == 0.0
    assert bool(out[0, 4].isnan()) and float(out[0, 5]) == math.inf
    out = rules.apply(x, masks=dev([[0b101010]]))
    assert out.cpu().tolist()[0] == [-math.inf, -math.inf, -math.inf, 0.0, -math.inf, math.inf]


def test_long_histories_count_exactly():
    n = 100000
    h = torch.zeros((1, n), dtype=torch.int32, device="cuda")
    h[0, ::3] = 5
    rules = pkg.TokenRules(9, h, dev([n]), counted_from=dev([10]), frequency=f32([1.0]))
    out = rules.apply(torch.zeros((1, 9), device="cuda"))
    rules.check()
    host = h.cpu().numpy()[0, 10:]
    assert out.cpu().tolist()[0] == [-float((host == v).sum()) for v in range(9)]


@pytest.mark.parametrize("bad", ["seq", "negative seq", "len", "mask", "tree", "large tree", "starts", "bias"])
def test_bad_rows_are_reported_and_left(bad):
    V = 100
    bias = (dev([0, 1, 2, 3]), dev([1, 2, 3]), f32([1, 1, 1]))
    lens = dev([4, 4, 4])
    rules = pkg.TokenRules(V, dev(np.zeros((3, 8))), lens, frequency=f32([1, 1, 1]), bias=bias)
    logits = torch.zeros((200, V), device="cuda")
    out = torch.full((200, V), 3.0, device="cuda")
    seqs, starts = [0, 1, 2], [0, 60, 120, 180]
    parents = sum(([tree_ref.chain(60) for _ in range(3)]), []) + [0] * 20
    which = [0] * 200
    hit = slice(60, 120)
    if bad == "seq":
        seqs[1] = 3
    elif bad == "negative seq":
        seqs[1] = -1
    elif bad == "len":
        lens[1] = 9
    elif bad == "mask":
        which[60:120] = [1] * 30 + [-2] * 30
    elif bad == "tree":
        parents[70] = 10
    elif bad == "large tree":
        starts = [0, 60, 130, 190]
        parents = [-1] * 200
        hit = slice(60, 130)
    elif bad == "starts":
        starts = [60, 120, 180, 180]
        hit = slice(0, 60)
    else:
        bias[0][1], bias[0][2] = 2, 1
    rules.apply(logits, seqs=dev(seqs), starts=dev(starts), parents=dev(parents), drafted=dev([7] * 200), masks=dev([[-1] * 4]), mask_rows=dev(which), out=out)
    with pytest.raises(pkg.L2Error, match="invalid"):
        rules.check()
    assert bool((out[hit] == 3.0).all())
    last = 190 if bad == "large tree" else 180
    assert bool((out[last:] == 3.0).all())
    good = torch.ones(200, dtype=torch.bool)
    good[hit] = False
    good[last:] = False
    if bad == "bias":
        good[0:60] = True
    assert bool((out[good.cuda()][:, 0] == -4.0).all())
    rules.check()   # the status was cleared


def test_a_graph_follows_histories_and_a_stream_keeps_its_arguments():
    V = 2000
    m = Made(V, 3, 50, 8)
    logits = torch.randn((3, V), device="cuda")
    which, masks = dev([0, 1, 2]), m.packed()
    out = torch.empty((3, V), device="cuda")
    m.rules.apply(logits, masks=masks, mask_rows=which, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.rules.apply(logits, masks=masks, mask_rows=which, out=out)
    for turn in range(3):
        logits.normal_()
        m.lens = m.rng.integers(0, 51, 3)
        m.history = m.rng.integers(0, V, (3, 50))
        m.rules._kept[1].copy_(dev(m.lens))
        m.rules._kept[0].copy_(dev(m.history))
        which.copy_(dev([turn, 4, -1]))
        graph.replay()
        m.rules.check()
        for r, w in enumerate([turn, 4, None]):
            check(out[r], *m.row(logits[r].double().cpu().numpy(), r, [], w))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        mine = [t.clone() for t in (logits, which, masks)]
    got = m.rules.apply(mine[0], masks=mine[2], mask_rows=mine[1], stream=st)
    del mine
    torch.empty(3 * V, device="cuda").fill_(1e9)
    torch.cuda.synchronize()
    assert torch.equal(got, out)


def test_a_masked_row_is_sampled():
    """Rows of -inf (a mask that allows nothing) and rows that one token is left of, at any temperature."""
    V = 500
    rules = pkg.TokenRules(V, dev(np.zeros((3, 1))), dev([0, 0, 0]))
    allowed = np.zeros((3, 16 * 32), np.uint8)
    allowed[1, 321] = 1
    allowed[2, [7, 400]] = 1
    masks = torch.from_numpy(np.packbits(allowed, axis=1, bitorder="little").view(np.int32).copy()).cuda()
    for temperature, topp in ((0.0, 0.0), (1.0, 0.0), (0.7, 0.9), (1.0, 1.0), (100.0, 0.5)):
        rng = torch.tensor([11, 12, 13], dtype=torch.int64, device="cuda")
        tokens = torch.full((3,), -5, dtype=torch.int32, device="cuda")
        pkg.sample(rules.apply(torch.randn((3, V), device="cuda"), masks=masks), temperature, topp, rng, out=tokens)
        assert tokens[0].item() == 0 and tokens[1].item() == 321 and tokens[2].item() in (7, 400)
        assert (rng.tolist() == [11, 12, 13]) == (temperature == 0.0)


def test_rules_the_host_refuses():
    hist, lens = dev(np.zeros((2, 4))), dev([1, 1])
    for args in ((10, hist.cpu(), lens), (10, hist.float(), lens), (10, hist[0], lens), (10, hist.t(), dev([1] * 4)), (10, hist, dev([1])), (10, hist, None)):
        with pytest.raises(ValueError):
            pkg.TokenRules(*args)
    for kw in (dict(repetition=dev([1, 1])), dict(presence=f32([1])), dict(counted_from=f32([0, 0])), dict(bias=(dev([0, 0, 1]), dev([1]))),
               dict(bias=(dev([0, 1]), dev([1]), f32([1]))), dict(bias=(dev([0, 0, 1]), dev([1]), f32([1, 2]))), dict(bias=(dev([0, 0, 1]), dev([1]), None))):
        with pytest.raises(ValueError):
            pkg.TokenRules(10, hist, lens, **kw)
    for V in (0, -1, (1 << 24) + 1):
        with pytest.raises(pkg.L2Error, match="vocab_size"):
            pkg.TokenRules(V, hist, lens)
    rules = pkg.TokenRules(64, hist, lens)
    x = torch.zeros((2, 64), device="cuda")
    assert rules.apply(x[:0]).shape == (0, 64)
    for kw in (dict(seqs=dev([0])), dict(parents=dev([0, 0])), dict(masks=dev([[0]])), dict(mask_rows=dev([0, 0])), dict(out=x[:1]),
               dict(out=torch.zeros((2, 64), device="cuda"), out_dtype=torch.bfloat16), dict(out_dtype=torch.float64), dict(drafted=dev([1])),
               dict(masks=torch.zeros((2, 4), dtype=torch.int32, device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            rules.apply(x, **kw)
    with pytest.raises(ValueError):
        rules.apply(x[:, :63])
    with pytest.raises(pkg.L2Error, match="out_dtype"):
        rules.apply(x, out_dtype=torch.bfloat16)
    with pytest.raises(pkg.L2Error, match="exceeds"):
        rules.apply(torch.zeros((3, 64), device="cuda"))
    with pytest.raises(pkg.L2Error, match="n_masks"):
        rules.apply(x, masks=dev([[0, 0]]))
    with pytest.raises(pkg.L2Error, match="out_row_stride"):
        rules.apply(x, out=torch.zeros((1, 64), device="cuda").expand(2, 64))
    flat = torch.zeros(300, device="cuda")
    with pytest.raises(pkg.L2Error, match="shares memory"):
        rules.apply(flat[:128].view(2, 64), out=flat[64:192].view(2, 64))
