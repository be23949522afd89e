"""Steps with drafted tokens, all operators together as a serving loop uses them: a small two-layer model whose keys live in a pool
generates the same tokens with trees of drafts as without."""
import numpy as np
import pytest

from tests import tree_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402
from tests.test_gpu_pages import dev  # noqa: E402

L, H, KV, HS, V, DIM = 2, 8, 2, 64, 997, 128


class Model:
    """Random weights whose logits have clear maxima; attention, positions and rules are the package's."""

    def __init__(self, n_seqs, dtype, layout):
        g = torch.Generator(device="cuda").manual_seed(7)
        mat = lambda *s: torch.randn(s, generator=g, device="cuda") / s[0] ** 0.5  # noqa: E731
        self.emb, self.head = mat(V, DIM) * 30, mat(DIM, V) * 4
        self.qkv, self.out = [mat(DIM, (H + 2 * KV) * HS) for _ in range(L)], [mat(H * HS, DIM) for _ in range(L)]
        self.dtype = dtype
        self.pool = pkg.PagePool(L, 600, KV, 16, HS, n_seqs, 40, dtype=dtype)
        self.rope = pkg.Rope(HS, layout=layout, kind="bands", factor=4.0, original_len=64.0, low=1.0, high=4.0)
        self.history = torch.zeros((n_seqs, 300), dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        ones = torch.ones(n_seqs, device="cuda")
        rng = np.random.default_rng(5)
        self.masks = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (3, -(-V // 32))).astype(np.int32)).cuda()
        self.rules = pkg.TokenRules(V, self.history, self.lens, repetition=1.3 * ones, presence=0.2 * ones, frequency=0.1 * ones,
                                    bias=(dev(np.arange(n_seqs + 1)), dev([3] * n_seqs), torch.full((n_seqs,), -1.0, device="cuda")))

    def step(self, tokens, seqs, starts, parents, depth, mask_rows):
        """Appends the tokens' rows and returns what follows each (greedy)."""
        trees = starts[1:] - starts[:-1]
        of = torch.repeat_interleave(torch.arange(len(seqs), device="cuda"), trees.long(), output_size=tokens.numel())
        positions = self.pool.lens[seqs.long()][of] + depth
        x = self.emb[tokens.long()]
        for layer in range(L):
            y = (x / x.norm(dim=1, keepdim=True) * DIM ** 0.5) @ self.qkv[layer]
            y = y.to(self.dtype).view(-1, H + 2 * KV, HS)
            q, k, v = y[:, :H], y[:, H:H + KV], y[:, H + KV:]
            self.rope.apply(positions, q, k, out_q=q, out_k=k)
            self.pool.append(k, v, seqs, starts, layer=layer)
            o = self.pool.tree_attention(q, layer, seqs, starts, parents=parents)
            x = x + o.float().reshape(-1, H * HS) @ self.out[layer]
        logits = self.rules.apply(x @ self.head, seqs=seqs, starts=starts, parents=parents, drafted=tokens, masks=self.masks, mask_rows=mask_rows)
        rng = torch.ones(tokens.numel(), dtype=torch.int64, device="cuda")
        return pkg.sample(logits, 0.0, 0.0, rng)

    def commit(self, seqs, kept):
        for s, toks in zip(seqs, kept):
            n = int(self.lens[s])
            self.history[s, n:n + len(toks)] = dev(toks)
            self.lens[s] = n + len(toks)


@pytest.mark.parametrize("dtype,layout", [(torch.float32, "interleaved"), (torch.bfloat16, "half")])
def test_drafts_give_the_same_tokens_in_fewer_steps(dtype, layout):
    n = 3
    prompts = [[5, 17, 400, 9], [800], [1, 2, 3, 4, 5, 6, 7]]
    mask_of = lambda s, step: (s + step) % 4 - 1  # noqa: E731   (a grammar that goes on with each token)

    # one token a step
    m = Model(n, dtype, layout)
    plain = [list(p) for p in prompts]
    fed = [0] * n
    for _ in range(40):
        last = dev([0] * n)
        while any(fed[s] < len(plain[s]) for s in range(n)):
            who = [s for s in range(n) if fed[s] < len(plain[s])]
            toks = [plain[s][fed[s]] for s in who]
            got = m.step(dev(toks), dev(who), dev(range(len(who) + 1)), None, dev([0] * len(who)), dev([mask_of(s, fed[s]) for s in who]))
            m.commit(who, [[t] for t in toks])
            last[torch.tensor(who, device="cuda")] = got
            for s in who:
                fed[s] += 1
        for s, t in enumerate(last.tolist()):
            plain[s].append(t)
    m.pool.check()
    m.rules.check()

    # trees of drafts: right ones for a while, beside wrong ones; prompts come in as chains
    m = Model(n, dtype, layout)
    drafted = [list(p) for p in prompts]
    rng = np.random.default_rng(1)
    steps = 0
    while min(len(d) for d in drafted) < len(plain[0]) - 10:
        trees, toks, depth = [], [], []
        for s in range(n):
            done = int(m.lens[s])
            first = drafted[s][done:]                             # known tokens that are not yet in the pool: a chain
            parents, mine = tree_ref.chain(len(first)), list(first)
            at = len(mine) - 1
            for _ in range(int(rng.integers(0, 5))):              # guesses: the right token after the last right one, with wrong siblings before and after
                nxt = plain[s][done + len(tree_ref.line(parents, at))] if done + len(tree_ref.line(parents, at)) < len(plain[s]) else 0
                wrong = int(rng.integers(0, 3))
                for t in [int(x) for x in rng.integers(0, V, wrong)] + [nxt]:
                    parents.append(at)
                    mine.append(t)
                if rng.random() < 0.8:
                    at = len(mine) - 1
            trees.append(parents)
            toks.append(mine)
            depth += [len(tree_ref.line(parents, u)) - 1 for u in range(len(parents))]
        starts = np.concatenate([[0], np.cumsum([len(t) for t in trees])])
        parents = dev(np.concatenate([np.array(t, int) for t in trees]))
        flat = dev([t for x in toks for t in x])
        base = [int(x) for x in m.lens.tolist()]
        masks = [mask_of(s, base[s] + len(tree_ref.line(trees[s], u)) - 1) for s in range(n) for u in range(len(trees[s]))]
        targets = m.step(flat, dev(range(n)), dev(starts), parents, dev(depth), dev(masks))
        # what is known already is accepted whatever the model says: its parents' targets are the known tokens
        known = targets.clone()
        for s in range(n):
            for u in range(len(drafted[s]) - base[s] - 1):
                known[int(starts[s]) + u] = toks[s][u + 1]
        path, counts, following = m.pool.accept(flat, known, dev(range(n)), dev(starts), parents=parents)
        steps += 1
        for s in range(n):
            got = path[int(starts[s]):int(starts[s]) + int(counts[s])].tolist()
            m.commit([s], [[toks[s][u] for u in got]])
            drafted[s] = drafted[s][:base[s]] + [toks[s][u] for u in got] + [int(following[s])]
        assert m.pool.lens.tolist() == m.lens.tolist()
    m.pool.check()
    m.rules.check()
    for s in range(n):
        k = min(len(plain[s]), len(drafted[s]))
        assert plain[s][:k] == drafted[s][:k], s
    assert steps < 30
    m.pool.free(dev(range(n)))
    m.pool.check()
    assert int(m.pool.refs.abs().sum()) == 0
