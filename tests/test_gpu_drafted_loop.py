"""A generation loop with drafted tokens that never asks the GPU anything: one step (rotary positions, append, attention, rules, sampling, acceptance,
histories) in one graph, replayed, against the same model one token at a time."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402
from tests.test_gpu_drafted_step import V, Model  # noqa: E402
from tests.test_gpu_pages import dev  # noqa: E402

N, ROOM = 3, 300
PROMPTS = [[5, 17, 400, 9], [800], [1, 2, 3, 4, 5, 6, 7]]
# a tree of seven: a chain of the guesses 0, 1, 2, 3 with a wrong sibling before and one after some of them
PARENTS, DEPTH, GUESS = [-1, 0, 0, 2, 2, 3, 5], [0, 1, 1, 2, 2, 3, 4], [True, False, True, True, False, True, True]
SIZE = len(PARENTS)


def model(dtype, layout):
    m = Model(N, dtype, layout)
    m.book = torch.zeros((N, ROOM + 1), dtype=torch.int32, device="cuda")     # the last column takes what is not kept
    ones = torch.ones(N, device="cuda")
    m.rules = pkg.TokenRules(V, m.book[:, :ROOM], m.lens, repetition=1.5 * ones, presence=0.3 * ones, frequency=0.4 * ones)
    return m


def masks_of(lens, seqs, depth):
    """A grammar that goes on with each token: rows of Model.masks, -1 for none."""
    return ((seqs + lens[seqs] + depth) % 4 - 1).int()


def prompts(m):
    """The prompts' rows, and the token that follows each."""
    seqs = torch.arange(N, device="cuda")
    following = torch.zeros(N, dtype=torch.int32, device="cuda")
    for i in range(max(map(len, PROMPTS))):
        who = [s for s in range(N) if i < len(PROMPTS[s])]
        toks = dev([PROMPTS[s][i] for s in who])
        one(m, toks, seqs[who], following)
    return following


def one(m, tokens, who, following):
    """A step of one token for each of some sequences."""
    n = len(who)
    got = m.step(tokens, who.int(), dev(range(n + 1)), None, dev([0] * n), masks_of(m.lens, who, 0))
    m.book[who, m.lens[who].long()] = tokens
    m.lens[who] += 1
    following[who] = got


class Loop:
    """One step of all sequences as tensors that stay where they are."""

    def __init__(self, m, following, script):
        self.m, self.script = m, script               # script [N][..]: what a draft model would say at each position
        self.seqs, self.starts = dev(range(N)), dev(np.arange(N + 1) * SIZE)
        self.tree = torch.arange(N, device="cuda").repeat_interleave(SIZE)      # of each row
        self.place = torch.arange(N * SIZE, device="cuda") % SIZE
        self.parents, self.depth = dev(PARENTS * N), dev(DEPTH * N)
        self.right = torch.tensor(GUESS * N, device="cuda")
        self.tokens = torch.zeros(N * SIZE, dtype=torch.int32, device="cuda")
        self.roots = self.starts[:-1].long()
        self.tokens[self.roots] = following
        self.steps = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step(self):
        m, tree, tokens = self.m, self.tree, self.tokens
        # drafts: the script's tokens, wrong ones beside them; every third step they go wrong from the second on
        guess = self.script[tree, (m.lens[tree] + self.depth).clamp(max=self.script.shape[1] - 1)]
        off = (~self.right) | ((self.steps % 3 == 2) & (self.depth >= 2))
        drafts = torch.where(off, (guess + 1 + self.place) % V, guess).int()
        root = tokens[self.roots]
        tokens.copy_(drafts)
        tokens[self.roots] = root
        targets = m.step(tokens, self.seqs, self.starts, self.parents, self.depth, masks_of(m.lens, tree, self.depth))
        path, counts, following = m.pool.accept(tokens, targets, self.seqs, self.starts, parents=self.parents)
        # the accepted tokens go into the histories, and what follows them is the next step's first; a refused step is tried again
        kept = tokens[self.roots[tree] + path.clamp(min=0)]
        m.book[tree, torch.where(path >= 0, m.lens[tree] + self.place, ROOM)] = kept
        m.lens += counts
        tokens[self.roots] = torch.where(counts > 0, following, root)
        self.steps += 1


@pytest.mark.parametrize("dtype,layout", [(torch.float32, "interleaved"), (torch.bfloat16, "half")])
def test_a_captured_step_generates_what_single_tokens_do(dtype, layout):
    # one token a step
    m = model(dtype, layout)
    following = prompts(m)
    for _ in range(70):
        one(m, following.clone(), torch.arange(N, device="cuda"), following)
    m.pool.check()
    m.rules.check()
    plain, total = m.book.clone(), int(m.lens.min())

    m = model(dtype, layout)
    loop = Loop(m, prompts(m), plain[:, :total].long())
    first = m.lens.clone()
    loop.step()                                        # loads what the capture needs
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step()
    for _ in range(14):
        graph.replay()
    m.pool.check()
    m.rules.check()
    assert torch.equal(m.pool.lens, m.lens)
    assert 15 * 2 <= int((m.lens - first).min()) and int(m.lens.max()) <= total + 7
    for s in range(N):
        n = min(int(m.lens[s]), total)
        assert m.book[s, :n].tolist() == plain[s, :n].tolist(), s
        assert int(loop.tokens[loop.roots[s]]) == int(plain[s, n]) or n == total

    # a pool that is full refuses steps; nothing is lost, and once there is room they go on
    free = (m.pool.refs == 0).nonzero()[:, 0]
    m.pool.refs[free] = 1
    before, root = [t.clone() for t in (m.pool.k, m.pool.v, m.pool.lens, m.lens, m.book[:, :ROOM])], loop.tokens[loop.roots].clone()
    refused = 0
    for _ in range(6):                                 # until the last pages are full, whole steps may fit
        if refused == 0:
            before, root = [t.clone() for t in (m.pool.k, m.pool.v, m.pool.lens, m.lens, m.book[:, :ROOM])], loop.tokens[loop.roots].clone()
        graph.replay()
        torch.cuda.synchronize()
        refused += int(m.pool.status) != 0
    assert refused
    with pytest.raises(pkg.L2Error, match="free pages"):
        m.pool.check()
    for a, b in zip(before, (m.pool.k, m.pool.v, m.pool.lens, m.lens, m.book[:, :ROOM])):
        assert torch.equal(a, b)
    assert torch.equal(root, loop.tokens[loop.roots])
    m.pool.refs[free] = 0
    for _ in range(3):
        graph.replay()
    m.pool.check()
    m.rules.check()
    assert torch.equal(m.pool.lens, m.lens)
    for s in range(N):
        n = min(int(m.lens[s]), total)
        assert m.book[s, :n].tolist() == plain[s, :n].tolist(), s
