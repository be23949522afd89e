"""Random histories of steps on a pool that is nearly full, several batches taking turns without a wait: appends layer by layer, acceptances, given
paths, forks, frees and compactions against a plain statement in which a sequence is the list of its rows.  What is refused changes nothing, and what
a sequence has committed is never another's or lost."""
import numpy as np
import pytest

from tests import pages_ref, tree_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402
from tests.test_gpu_pages import DT, dev, same_books  # noqa: E402

L, KV, HS = 3, 2, 8


class Plain:
    """Rows by number (None: one that a layer was left out of), books as tests/pages_ref.py keeps them, and each page's word on its sequence's last rows."""

    def __init__(self, n_pages, ps, n_seqs, max_pages):
        self.ref = pages_ref.RefPool(n_pages, ps, n_seqs, max_pages)
        self.rows = [[] for _ in range(n_seqs)]
        self.word = [0] * n_pages           # 1: refused; 2 + layer: left out from that layer on
        self.held_back = False              # the last extension was refused
        self.next = 1

    def end(self, s):
        return int(self.ref.table[s, self.ref.held(s) - 1]) if self.ref.lens[s] else -1

    def extend(self, seqs, counts):
        r = self.ref
        last = [self.end(s) for s in seqs]
        old = [(r.held(s), [int(r.table[s, r.held(s) - 1])] if r.lens[s] else []) for s in seqs]
        alone = [p >= 0 and r.refs[p] == 1 for p in last]
        if r.append(seqs, counts) is None:
            for s, c in zip(seqs, counts):
                if c and self.end(s) >= 0:
                    self.word[self.end(s)] = 1
            self.held_back = True
            return False
        for s, c, p, a, (h, _) in zip(seqs, counts, last, alone, old):
            for j in range(h, r.held(s)):
                self.word[int(r.table[s, j])] = 0
            if c and a:
                self.word[p] = 0
            self.rows[s] += [[None] * L for _ in range(c)]
        self.held_back = False
        return True

    def write(self, seqs, counts, numbers, layer, extended):
        """Whether something was reported."""
        bad = False
        at = 0
        for s, c in zip(seqs, counts):
            mine = numbers[at:at + c]
            at += c
            p = self.end(s)
            if not c or (extended and self.held_back):
                continue
            if not extended:
                if self.held_back:
                    if p >= 0 and (self.word[p] == 0 or self.word[p] > 2 + layer):
                        self.word[p] = 2 + layer
                    continue
                if p >= 0 and self.word[p] == 1:
                    bad = True
                    continue
                if len(self.rows[s]) < c:
                    bad = True              # some of these rows have no place: the caller does not do that
                    continue
                if self.ref.refs[p] == 1 and self.word[p] > 1 and 2 + layer <= self.word[p]:
                    self.word[p] = 0
            base = len(self.rows[s]) - c
            for j, x in enumerate(mine):
                if not extended and self.ref.refs[self.ref.table[s, (base + j) // self.ref.ps]] != 1:
                    bad = True              # a fork holds the page, too
                else:
                    self.rows[s][base + j][layer] = x
        return bad

    def keep(self, seqs, sizes, paths):
        """Whether the call is done: all of it or nothing."""
        r, ps = self.ref, self.ref.ps
        for s, n, path in zip(seqs, sizes, paths):
            if len(self.rows[s]) < n:
                return False
            if not n:
                continue
            if self.word[self.end(s)]:
                return False
            c, base = len(path), len(self.rows[s]) - n
            if c == n:
                continue
            stay = next((i for i, x in enumerate(path) if x != i), c)
            now = base + c
            for col in range(base // ps, r.held(s)):
                moved = base + stay < now and base + stay < (col + 1) * ps and col * ps < now
                part = col * ps < now < (col + 1) * ps
                if (moved or part) and r.refs[r.table[s, col]] != 1:
                    return False
        for s, n, path in zip(seqs, sizes, paths):
            base = len(self.rows[s]) - n
            self.rows[s] = self.rows[s][:base] + [self.rows[s][base + j] for j in path]
            for col in range(-(-len(self.rows[s]) // ps), r.held(s)):
                r.refs[r.table[s, col]] -= 1
            r.lens[s] = len(self.rows[s])
        return True

    def fork(self, src, dst, counts):
        copies = self.ref.fork(src, dst, counts)
        if copies is None:
            return False
        for a, b, _ in copies:
            self.word[b] = self.word[a]
        for s, d, c in zip(src, dst, counts):
            self.rows[d] = [list(x) for x in self.rows[s][:c]]
        return True

    def free(self, seqs, compact):
        for s in seqs:
            self.rows[s] = []
        moves = self.ref.free(seqs, compact)
        word = list(self.word)
        for a, b in moves:
            self.word[b] = word[a]


def value(numbers, layer, dtype):
    """The row of a number in a layer, [rows][heads][head size]: different in each, exact in every type."""
    n = torch.tensor([x or 0 for x in numbers], device="cuda", dtype=torch.float32)
    e = torch.arange(KV * HS, device="cuda", dtype=torch.float32).view(KV, HS)
    return ((n[:, None, None] * 7 + e * 3 + layer * 5) % 251 - 125).to(dtype)


def compare(pool, plain):
    same_books(pool, plain.ref)
    for s, rows in enumerate(plain.rows):
        n = len(rows)
        if not n:
            continue
        t = plain.ref.table[s]
        page = torch.tensor([int(t[i // pool.page_size]) for i in range(n)], device="cuda")
        at = torch.tensor([i % pool.page_size for i in range(n)], device="cuda")
        for layer in range(L):
            known = torch.tensor([r[layer] is not None for r in rows], device="cuda")
            want = value([r[layer] for r in rows], layer, pool.dtype)
            k, v = (x[layer].permute(0, 2, 1, 3)[page, at] for x in (pool.k, pool.v))
            assert torch.equal(k[known], want[known]) and torch.equal(v[known], -want[known]), (s, layer)


@pytest.mark.parametrize("dtype,ps,n_pages,seed", [
    ("fp32", 4, 20, 0), ("bf16", 8, 14, 1), ("fp16", 1, 45, 2), ("fp32", 16, 9, 3), ("bf16", 5, 17, 4), ("fp32", 8, 14, 5), ("fp16", 4, 25, 6), ("bf16", 2, 40, 7)])
def test_histories_with_refusals(dtype, ps, n_pages, seed):
    rng = np.random.default_rng(seed)
    n_seqs, max_pages = 7, -(-60 // ps)
    pool = pkg.PagePool(L, n_pages, KV, ps, HS, n_seqs, max_pages, dtype=DT[dtype])
    plain = Plain(n_pages, ps, n_seqs, max_pages)
    open_steps = []                          # batches under way: [seqs, sizes, numbers, layers still to write, extended]
    seen = dict.fromkeys(("append", "no append", "accept", "no accept", "fork", "no fork"), 0)

    def status(expected):
        if expected:
            with pytest.raises(pkg.L2Error):
                pool.check()
        else:
            pool.check()

    for turn in range(220):
        op = rng.choice(["step", "step", "layer", "layer", "layer", "accept", "accept", "fork", "free"], p=None)
        if op == "step" and len(open_steps) < 2:
            busy = {s for st in open_steps for s in st["seqs"]}
            seqs = [int(s) for s in rng.permutation(n_seqs) if s not in busy][:int(rng.integers(1, 4))]
            if not seqs:
                continue
            sizes = [int(rng.integers(0, 2 * ps + 6)) for _ in seqs]
            numbers = list(range(plain.next, plain.next + sum(sizes)))
            plain.next += len(numbers)
            ok = plain.extend(seqs, sizes)
            plain.write(seqs, sizes, numbers, 0, True)
            x = value(numbers, 0, DT[dtype])
            pool.append(x, -x, dev(seqs), dev(np.concatenate([[0], np.cumsum(sizes)])), layer=0)
            status(not ok)
            seen["append" if ok else "no append"] += 1
            open_steps.append(dict(seqs=seqs, sizes=sizes, numbers=numbers, layers=list(range(1, L))))
        elif op == "layer" and any(st["layers"] for st in open_steps):
            st = rng.choice([st for st in open_steps if st["layers"]])
            layer = st["layers"].pop(0)
            if any(c > len(plain.rows[s]) for s, c in zip(st["seqs"], st["sizes"])):
                continue                     # rows without a place are no subject here
            bad = plain.write(st["seqs"], st["sizes"], st["numbers"], layer, False)
            x = value(st["numbers"], layer, DT[dtype])
            pool.append(x, -x, dev(st["seqs"]), dev(np.concatenate([[0], np.cumsum(st["sizes"])])), layer=layer)
            status(bad)
        elif op == "accept" and open_steps:
            st = open_steps.pop(int(rng.integers(0, len(open_steps))))
            if any(st["layers"]) and rng.random() < 0.7:
                open_steps.append(st)
                continue
            sizes = [min(n, 64) for n in st["sizes"]]
            starts = np.concatenate([[0], np.cumsum(sizes)])
            if rng.random() < 0.5:
                trees = [tree_ref.random_tree(rng, n, back=3) for n in sizes]
                tar = [[int(x) for x in rng.integers(0, 9, n)] for n in sizes]
                tok = [[tar[i][p] if p >= 0 and rng.random() < 0.8 else 3 for p in t] for i, t in enumerate(trees)]
                want = [tree_ref.accepted(t, a, b) for t, a, b in zip(trees, tok, tar)]
                done = plain.keep(st["seqs"], sizes, [w[0] for w in want])
                flat = lambda v: dev([x for y in v for x in y])  # noqa: E731
                path, counts, following = pool.accept(flat(tok), flat(tar), dev(st["seqs"]), dev(starts), parents=flat(trees))
                status(not done)
                assert counts.tolist() == ([len(w[0]) for w in want] if done else [0] * len(sizes))
                assert following.tolist() == ([w[1] for w in want] if done else [-1] * len(sizes))
                assert path.tolist() == ([x for w, n in zip(want, sizes) for x in w[0] + [-1] * (n - len(w[0]))] if done else [-1] * int(starts[-1]))
            else:
                paths = [sorted(int(x) for x in rng.choice(n, rng.integers(0, n + 1), replace=False)) if n else [] for n in sizes]
                done = plain.keep(st["seqs"], sizes, paths)
                pool.keep(dev([x for p, n in zip(paths, sizes) for x in p + [0] * (n - len(p))]), dev([len(p) for p in paths]), dev(st["seqs"]), dev(starts))
                status(not done)
            seen["accept" if done else "no accept"] += 1
        elif op == "fork":
            busy = {s for st in open_steps for s in st["seqs"]}
            empty = [s for s in range(n_seqs) if not plain.rows[s] and s not in busy]
            full = [s for s in range(n_seqs) if plain.rows[s]]
            if not empty or not full or rng.random() < 0.4:
                continue
            src, dst = int(rng.choice(full)), int(rng.choice(empty))
            count = int(rng.integers(1, len(plain.rows[src]) + 1)) if rng.random() < 0.5 else len(plain.rows[src])
            ok = plain.fork([src], [dst], [count])
            pool.fork(dev([src]), dev([dst]), dev([count]))
            status(not ok)
            seen["fork" if ok else "no fork"] += 1
        elif op == "free" and rng.random() < 0.5:
            busy = {s for st in open_steps for s in st["seqs"]}
            seqs = [int(s) for s in rng.permutation(n_seqs) if s not in busy][:int(rng.integers(0, 3))]
            compact = bool(rng.random() < 0.6)
            plain.free(seqs, compact)
            pool.free(dev(seqs) if seqs else None, compact=compact)
            status(False)
        compare(pool, plain)
    assert min(seen["append"], seen["accept"], seen["fork"], seen["no append"] + seen["no accept"]) >= 3, seen
