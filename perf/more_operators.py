"""Measured cases of the operators of a step with drafted tokens: rotary
positions of its queries and keys, attention of trees of drafted tokens over a
page pool, the rules on its logits (penalties, biases, grammar masks), and the
acceptance of a path of each tree with the pool shortened to it.

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, through the package.

A sequence holds its committed rows and, behind them, one row for each drafted
token of its tree; ``parents`` gives each token's parent within its own tree
(-1: it hangs on the committed rows; no array: a chain).  ``starts`` bounds the
trees within the call's rows.  Pools are laid out, and their pages shuffled, as
in a pool that has served for a while.
"""
import math
import zlib

import numpy as np
import torch

own = False

_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_SIZES = {"fp32": 4, "bf16": 2, "fp16": 2}


# --------------------------------------------------------------------------
# cases

def listed():
    return [
        # a small model with one user and a tree of seven tokens (latency of one call)
        dict(name="tree_tiny_fp32", op="attn", dtype="fp32", heads=8, kv=4, hs=8, page=16, seqs=1, tree="wide",
             nodes_lo=7, nodes_hi=7, prefix_lo=100, prefix_hi=100),
        # a mid-size model, eight chats of different lengths, trees of 16 tokens
        dict(name="tree_mid_bf16", op="attn", dtype="bf16", heads=12, kv=12, hs=64, page=16, seqs=8, tree="wide",
             nodes_lo=16, nodes_hi=16, prefix_lo=0, prefix_hi=1001),
        # grouped heads, 16 sequences, the largest trees: 512 (token, head) pairs on a KV head
        dict(name="tree_gqa_fp16", op="attn", dtype="fp16", heads=32, kv=4, hs=64, page=32, seqs=16, tree="wide",
             nodes_lo=60, nodes_hi=64, prefix_lo=500, prefix_hi=4000),
        # the 7B head shape over an fp32 cache, ragged trees
        dict(name="tree_7b_fp32", op="attn", dtype="fp32", heads=32, kv=32, hs=128, page=64, seqs=8, tree="deep",
             nodes_lo=1, nodes_hi=26, prefix_lo=1000, prefix_hi=3001),
        # chains of five tokens for each of 64 long chats, grouped heads: what a draft model or an n-gram table proposes
        dict(name="chain_gqa_bf16_long", op="attn", dtype="bf16", heads=32, kv=8, hs=128, page=32, seqs=64, tree="chain",
             nodes_lo=5, nodes_hi=5, prefix_lo=1000, prefix_hi=8190),
        # a small model's tree of seven, up to three tokens accepted
        dict(name="accept_tiny_fp32", op="accept", dtype="fp32", layers=5, kv=4, hs=8, page=16, seqs=1, nodes_lo=7, nodes_hi=7,
             most=3, prefix_lo=100, prefix_hi=100),
        # the 7B shape, 16 sequences with trees of up to 64 tokens, up to nine accepted, every layer's rows moved
        dict(name="accept_7b_bf16", op="accept", dtype="bf16", layers=32, kv=32, hs=128, page=16, seqs=16, nodes_lo=40, nodes_hi=64,
             most=9, prefix_lo=1, prefix_hi=90),
        # one user of a small model, every rule at once (latency of one call)
        dict(name="rules_tiny_fp32", op="rules", dtype="fp32", vocab=512, seqs=1, nodes_lo=1, nodes_hi=1, drafted=False, hist_lo=40,
             hist_hi=40, penalties=True, bias=5, masks=True),
        # a batch of 64 with long histories, an odd vocabulary
        dict(name="rules_batch_fp32", op="rules", dtype="fp32", vocab=32003, seqs=64, nodes_lo=1, nodes_hi=1, drafted=False, hist_lo=1,
             hist_hi=4000, penalties=True, bias=20, masks=True),
        # logits of 16 trees as a 16-bit classifier leaves them: each token's own path counts, and each has its own mask
        dict(name="rules_trees_bf16", op="rules", dtype="bf16", vocab=128000, seqs=16, nodes_lo=20, nodes_hi=40, drafted=True,
             hist_lo=100, hist_hi=8000, penalties=True, bias=0, masks=True),
        # one step's queries and keys of 64 sequences, neighbours as pairs
        dict(name="rope_step_bf16", op="rope", dtype="bf16", heads=32, kv=8, hs=128, rot=128, rows=64, half=False, scaling="plain",
             far=8192),
        # a packed prompt at far positions, halves as pairs in half of each head, scaled by wavelength
        dict(name="rope_prompt_fp16", op="rope", dtype="fp16", heads=32, kv=4, hs=64, rot=32, rows=16384, half=True, scaling="bands",
             far=1000000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# (query heads, KV heads, head size): the decoder's shapes
_HEADS = [(8, 4, 8), (6, 4, 48), (12, 12, 64), (32, 4, 64), (32, 32, 128), (32, 8, 128), (16, 2, 64), (8, 1, 128)]


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "accept", "rules", "rules", "rope"])
    dtype = rng.choice(["fp32", "bf16", "fp16"])
    heads, kv, hs = rng.choice(_HEADS)
    page = rng.choice([16, 24, 32, 64, 128])
    if op == "attn":
        seqs = _log_int(rng, 1, 64)
        nodes = _log_int(rng, 1, min(64, 1024 // seqs))
        # keys of all sequences together, padded: within what the plain form holds
        top = min(8000, max(16, int((2.0e8 if dtype == "fp32" else 4.0e8) / (seqs * kv * hs))))
        hi = _log_int(rng, 16, top)
        return dict(op=op, dtype=dtype, heads=heads, kv=kv, hs=hs, page=page, seqs=seqs, tree=rng.choice(["wide", "deep", "chain"]),
                    nodes_lo=rng.randint(1, nodes), nodes_hi=nodes, prefix_lo=rng.choice([0, hi // 2, hi]), prefix_hi=hi)
    if op == "accept":
        # whole pools are compared: about 1 GB at most
        layers, seqs = rng.randint(2, 32), _log_int(rng, 1, 64)
        room = int(1.0e9 / (2 * layers * kv * hs * _SIZES[dtype])) // seqs - page
        nodes = min(_log_int(rng, 1, 64), max(1, room // 2))
        return dict(op=op, dtype=dtype, layers=layers, kv=kv, hs=hs, page=page, seqs=seqs, nodes_lo=rng.randint(1, nodes), nodes_hi=nodes,
                    most=rng.randint(1, 12), prefix_lo=0, prefix_hi=_log_int(rng, 1, max(1, min(300, room - nodes))))
    if op == "rules":
        vocab = _log_int(rng, 500, 128000)
        seqs = _log_int(rng, 1, 64)
        nodes = _log_int(rng, 1, max(1, min(64, 512 // seqs, int(4.0e7 / (seqs * vocab)))))
        return dict(op=op, dtype=dtype, vocab=vocab, seqs=seqs, nodes_lo=rng.randint(1, nodes), nodes_hi=nodes,
                    drafted=nodes > 1 or rng.random() < 0.3, hist_lo=rng.choice([0, 1, 20]), hist_hi=_log_int(rng, 20, 8000),
                    penalties=rng.random() < 0.8, bias=rng.choice([0, 0, 3, 40]), masks=rng.random() < 0.7)
    rot = 2 * rng.randint(1, hs // 2) if rng.random() < 0.5 else hs
    most = max(2, int(4.0e7 / ((heads + kv) * hs)))
    return dict(op=op, dtype=dtype, heads=heads, kv=kv, hs=hs, rot=rot, rows=_log_int(rng, 1, min(16384, most)), half=rng.random() < 0.5,
                scaling=rng.choice(["plain", "linear", "base", "bands"]), far=_log_int(rng, 100, 1000000))


# --------------------------------------------------------------------------
# inputs

def _sizes(case):
    """The case's ragged sizes, which are the same for every seed: rows committed and drafted (or counted) of each sequence."""
    rng = np.random.default_rng(zlib.crc32(repr(sorted((a, b) for a, b in case.items() if a != "name")).encode()))
    nodes = rng.integers(case["nodes_lo"], case["nodes_hi"] + 1, case["seqs"])
    lo, hi = ("hist_lo", "hist_hi") if case["op"] == "rules" else ("prefix_lo", "prefix_hi")
    return rng.integers(case[lo], case[hi] + 1, case["seqs"]), nodes


def _tree(kind, n, rng):
    """Parents of n tokens: each token's parent comes before it.  wide: a few tokens with many children, as top-k drafts have;
    deep: long branches; chain: one."""
    back = {"wide": lambda i: int(i * rng.uniform(0.1, 0.9)), "deep": lambda i: max(0, i - int(rng.integers(1, 4))), "chain": lambda i: i - 1}[kind]
    return np.array([-1] + [back(i) for i in range(1, n)], np.int64)


def _accepted_tree(n, most, rng):
    """Parents, and the tokens that will be accepted.  Which ones those are is chosen so that a pass leaves the rows that it reads as
    they were (the j-th accepted one is token j, or comes behind all rows that accepted ones move to): passes then repeat one another."""
    c = int(rng.integers(1, min(most, n) + 1))
    stay = int(rng.integers(1, c + 1)) if n >= 2 * c else c
    path = list(range(stay)) + sorted(rng.choice(np.arange(c, n), c - stay, replace=False).tolist() if c > stay else [])
    parents = np.array([-1] + [int(rng.integers(0, i)) for i in range(1, n)], np.int64)
    for a, b in zip(path, path[1:]):
        parents[b] = a
    return parents, path


def _pool(case, lens, rng):
    """Counts and tables of a pool whose sequences hold `lens` rows in pages in no order."""
    ps = case["page"]
    held = -(-lens // ps)
    n_pages, width = int(held.sum()) + 3, int(held.max()) + 1
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    at = 0
    for s, h in enumerate(held):
        table[s, :h] = ids[at:at + h]
        refs[table[s, :h]] = 1
        at += h
    return refs, table


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=_DTYPES[case["dtype"]]):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    return {"attn": _prepare_pool, "accept": _prepare_pool, "rules": _prepare_rules, "rope": _prepare_rope}[case["op"]](case, rng, normal)


def _prepare_pool(case, rng, normal):
    prefix, nodes = _sizes(case)
    n, lens = case["seqs"], prefix + nodes
    starts = np.concatenate([[0], np.cumsum(nodes)])
    refs, table = _pool(case, lens, rng)
    layers = case.get("layers", 1)
    shape = (len(refs), case["kv"], case["page"], case["hs"])
    k, v = (torch.empty((layers, *shape), dtype=_DTYPES[case["dtype"]], device="cuda") for _ in range(2))
    for t in (k, v):
        for i in range(layers):
            t[i] = normal(*shape)
    # one block of integers: counts and lengths (so a pass can start from the same bookkeeping)
    book0 = _dev(np.concatenate([refs, lens]))
    book = book0.clone()
    st = dict(case=case, k=k, v=v, book0=book0, book=book, refs=book[:len(refs)], lens=book[len(refs):], table=_dev(table),
              seqs=_dev(rng.permutation(n)), starts=None, host=dict(prefix=prefix, nodes=nodes, table=table, refs=refs))
    # trees in the order of the call's sequences
    order = st["seqs"].cpu().numpy()
    mine = nodes[order]
    starts = np.concatenate([[0], np.cumsum(mine)])
    st["starts"] = _dev(starts)
    st["rows"], st["widest"] = int(starts[-1]), int(mine.max())
    if case["op"] == "attn":
        trees = [_tree(case["tree"], int(m), rng) for m in mine]
        st["parents"] = None if case["tree"] == "chain" else _dev(np.concatenate(trees))
        # queries that concentrate on some keys, as trained heads do
        st["q"] = normal(st["rows"], case["heads"], case["hs"], std=2.0)
        st["host"].update(order=order, starts=starts, trees=trees)
    else:
        vocab = 32000
        targets = rng.integers(0, vocab, st["rows"])   # what the model says follows each drafted token
        tokens = np.zeros(st["rows"], np.int64)
        trees, paths = [], []
        for a, m in zip(starts, mine):
            parents, path = _accepted_tree(int(m), case["most"], rng)
            right = np.isin(np.arange(m), path)
            above = targets[a + np.maximum(parents, 0)]
            tokens[a:a + m] = np.where(right, above, (above + rng.integers(1, vocab, m)) % vocab)
            trees.append(parents)
            paths.append(path)
        st["parents"] = _dev(np.concatenate(trees))
        st["tokens"], st["targets"] = _dev(tokens), _dev(targets)
        st["host"].update(order=order, starts=starts, trees=trees, paths=paths, targets=targets)
    if own:
        import llama_transformer_decode_gb300 as pkg
        st["pool"] = pkg.PagePool.from_tensors(k, v, refs=st["refs"], lens=st["lens"], table=st["table"])
    return st


def _prepare_rules(case, rng, normal):
    hist, nodes = _sizes(case)
    n, V = case["seqs"], case["vocab"]
    starts = np.concatenate([[0], np.cumsum(nodes)])
    rows = int(starts[-1])
    # tokens as text has them: few often, many seldom
    often = lambda *shape: np.minimum((V * rng.random(shape) ** 4).astype(np.int64), V - 1)  # noqa: E731
    st = dict(case=case, rows=rows, widest=int(nodes.max()), logits=normal(rows, V, std=3.0), history=_dev(often(n, int(hist.max()) + 1)),
              lens=_dev(hist), starts=_dev(starts), counted_from=_dev(hist // 3), seqs=_dev(np.arange(n)))
    trees = [_tree("wide", int(m), rng) for m in nodes]
    st["parents"] = _dev(np.concatenate(trees))
    st["drafted"] = _dev(often(rows)) if case["drafted"] else None
    st["repetition"] = st["presence"] = st["frequency"] = st["bias"] = st["masks"] = st["mask_rows"] = None
    f32 = lambda lo, hi: torch.from_numpy(rng.uniform(lo, hi, n).astype(np.float32)).cuda()  # noqa: E731
    if case["penalties"]:
        st["repetition"], st["presence"], st["frequency"] = f32(1.0, 1.3), f32(-0.5, 1.0), f32(0.0, 0.6)
    if case["bias"]:
        counts = rng.integers(0, case["bias"] + 1, n)
        tokens = [rng.choice(V, c, replace=False) for c in counts]
        st["bias"] = (_dev(np.concatenate([[0], np.cumsum(counts)])), _dev(np.concatenate(tokens)),
                      torch.from_numpy(rng.normal(0, 4, int(counts.sum())).astype(np.float32)).cuda())
    if case["masks"]:
        # grammars that allow little, half or nearly all, and one that allows nothing; some rows have none
        words = -(-V // 32)
        bits = rng.integers(0, 1 << 32, (8, words), dtype=np.uint32)
        bits[0] &= rng.integers(0, 1 << 32, words, dtype=np.uint32) & rng.integers(0, 1 << 32, words, dtype=np.uint32)
        bits[1] |= rng.integers(0, 1 << 32, words, dtype=np.uint32) | rng.integers(0, 1 << 32, words, dtype=np.uint32)
        bits[2] = 0
        st["masks"], st["mask_rows"] = torch.from_numpy(bits.view(np.int32)).cuda(), _dev(rng.integers(-1, 8, rows))
    st["host"] = dict(hist=hist, starts=starts, trees=trees)
    if own:
        import llama_transformer_decode_gb300 as pkg
        st["rules"] = pkg.TokenRules(V, st["history"], st["lens"], counted_from=st["counted_from"], repetition=st["repetition"],
                                     presence=st["presence"], frequency=st["frequency"], bias=st["bias"])
    return st


_SCALING = {  # what a model's configuration holds
    "plain": {},
    "linear": dict(kind="linear", factor=4.0),
    "base": dict(kind="base", factor=8.0),
    "bands": dict(kind="bands", factor=8.0, original_len=8192.0, low=1.0, high=4.0, amplitude=1.1),
}


def _prepare_rope(case, rng, normal):
    rows, hs = case["rows"], case["hs"]
    # queries, keys and values side by side, as one projection leaves them
    both = normal(rows, case["heads"] + 2 * case["kv"], hs)
    st = dict(case=case, q=both[:, :case["heads"]], k=both[:, case["heads"]:case["heads"] + case["kv"]], scaling=_SCALING[case["scaling"]],
              positions=_dev(rng.integers(0, case["far"] + 1, rows)))
    if own:
        import llama_transformer_decode_gb300 as pkg
        st["rope"] = pkg.Rope(case["rot"], base=10000.0, layout="half" if case["half"] else "interleaved", **st["scaling"])
    return st


# --------------------------------------------------------------------------
# one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    op = st["case"]["op"]
    if op == "attn":
        return st["pool"].tree_attention(st["q"], 0, st["seqs"], st["starts"], parents=st["parents"])
    if op == "accept":
        st["book"].copy_(st["book0"])
        path, counts, following = st["pool"].accept(st["tokens"], st["targets"], st["seqs"], st["starts"], parents=st["parents"])
        return dict(path=path, counts=counts, next=following, refs=st["refs"], lens=st["lens"], k=st["k"], v=st["v"])
    if op == "rules":
        return st["rules"].apply(st["logits"], seqs=st["seqs"], starts=st["starts"], parents=st["parents"], drafted=st["drafted"],
                                 masks=st["masks"], mask_rows=st["mask_rows"], out_dtype=torch.float32)
    q, k = st["rope"].apply(st["positions"], st["q"], st["k"])
    return dict(q=q, k=k)


def _run_plain(st):
    return {"attn": _plain_attention, "accept": _plain_accept, "rules": _plain_rules, "rope": _plain_rope}[st["case"]["op"]](st)


def _places(st):
    """Of each row, its tree and its place in it; of each tree, its first row and tokens."""
    starts = st["starts"].long()
    r = torch.arange(st["rows"], device="cuda")
    tree = torch.searchsorted(starts, r, right=True) - 1
    return tree, r - starts[tree], starts[:-1], starts[1:] - starts[:-1]


def _padded_parents(st):
    """Parents [trees][widest], -1 behind a tree's end."""
    tree, place, first, _ = _places(st)
    parents = torch.full((first.numel(), st["widest"]), -1, dtype=torch.long, device="cuda")
    parents[tree, place] = place - 1 if st["parents"] is None else st["parents"].long()
    return parents


def _ancestors(parents):
    """Whether token j is i or above it: [trees][widest i][widest j]."""
    w = parents.shape[1]
    ids = torch.arange(w, device="cuda")
    reach = ((parents[:, :, None] == ids) | (ids[:, None] == ids)).float()
    step = 1
    while step < w:   # paths of twice the length
        reach = (torch.matmul(reach, reach) > 0).float()
        step *= 2
    return reach > 0


def _plain_attention(st):
    case, ps = st["case"], st["case"]["page"]
    H, KV, hs = case["heads"], case["kv"], case["hs"]
    tree, place, first, count = _places(st)
    n, w = first.numel(), st["widest"]
    T = int((st["host"]["prefix"] + st["host"]["nodes"]).max())
    seqs = st["seqs"].long()
    lens = st["lens"].long()[seqs]
    pos = torch.arange(T, device="cuda")
    held = pos < lens[:, None]
    page = torch.where(held, st["table"].long()[seqs][:, pos // ps], 0)
    k = st["k"][0][page, :, pos % ps].transpose(1, 2).float()   # [n][kv][T][hs]
    v = st["v"][0][page, :, pos % ps].transpose(1, 2).float()
    # the query heads of each KV head, as many for each (the last one again where there are fewer)
    of = torch.arange(H, device="cuda") * KV // H
    gq = -(-H // KV)
    lead = torch.searchsorted(of, torch.arange(KV, device="cuda"))
    size = torch.bincount(of, minlength=KV)
    heads = lead[:, None] + torch.minimum(torch.arange(gq, device="cuda"), size[:, None] - 1)          # [kv][gq]
    row = first[:, None] + torch.minimum(torch.arange(w, device="cuda"), (count - 1)[:, None])         # [n][w]
    q = st["q"].float()[row][:, :, heads].permute(0, 2, 1, 3, 4).reshape(n, KV, w * gq, hs)
    s = torch.matmul(q, k.transpose(2, 3)).view(n, KV, w, gq, T) / math.sqrt(hs)
    # committed rows, and the token itself with those above it
    drafted = pos - (lens - count)[:, None]                                                            # [n][T]
    above = torch.gather(_ancestors(_padded_parents(st)), 2, drafted.clamp(0, w - 1)[:, None].expand(n, w, T))
    seen = held[:, None] & ((drafted < 0)[:, None] | above)
    s = torch.where(seen[:, None, :, None], s, -math.inf)
    e = torch.exp(s - s.max(dim=-1, keepdim=True).values)
    o = torch.matmul(e.view(n, KV, w * gq, T), v).view(n, KV, w, gq, hs) / e.sum(dim=-1, keepdim=True)
    h = torch.arange(H, device="cuda")
    return o[tree[:, None], of[h], place[:, None], h - lead[of]].to(st["q"].dtype)


def _plain_accept(st):
    case, ps = st["case"], st["case"]["page"]
    st["book"].copy_(st["book0"])
    refs, lens, table = st["refs"], st["lens"], st["table"].long()
    tree, place, first, count = _places(st)
    parents, seqs = _padded_parents(st), st["seqs"].long()
    n, w = parents.shape
    ids = torch.arange(w, device="cuda")
    there = ids < count[:, None]
    at = (first[:, None] + ids).clamp(max=st["rows"] - 1)
    tokens = torch.where(there, st["tokens"].long()[at], -1)
    targets = st["targets"].long()[at]
    # a token is chosen where it is what follows its parent and no sibling before it is; the first one always is
    right = there & (parents >= 0) & (tokens == torch.gather(targets, 1, parents.clamp(min=0)))
    older = (parents[:, :, None] == parents[:, None, :]) & (ids[:, None] > ids)
    chosen = right & ~(older & right[:, None, :]).any(dim=2)
    chosen[:, 0] = True
    # accepted: it and all above it are chosen
    accepted = there & ~(_ancestors(parents) & ~chosen[:, None, :]).any(dim=2)
    counts = accepted.sum(dim=1)
    order = torch.sort((~accepted).int(), dim=1, stable=True).indices
    kept = ids < counts[:, None]
    path = torch.where(kept, order, -1)[tree, place].int()
    following = targets[torch.arange(n, device="cuda"), order.gather(1, (counts - 1)[:, None])[:, 0]].int()
    # bookkeeping, and the rows of accepted tokens side by side
    old = lens[seqs].long()
    base, now = old - count, old - count + counts
    cols = torch.arange(table.shape[1], device="cuda")
    gone = (cols >= ((now + ps - 1) // ps)[:, None]) & (cols < ((old + ps - 1) // ps)[:, None])
    refs.index_add_(0, torch.where(gone, table[seqs], 0).reshape(-1), -gone.reshape(-1).int())
    lens[seqs] = now.int()
    i, j = torch.nonzero(kept, as_tuple=True)
    src, dst = base[i] + order[i, j], base[i] + j
    for pool in (st["k"], st["v"]):
        rows = pool.permute(1, 3, 0, 2, 4)
        rows[table[seqs[i], dst // ps], dst % ps] = rows[table[seqs[i], src // ps], src % ps]
    return dict(path=path, counts=counts.int(), next=following, refs=refs, lens=lens, k=st["k"], v=st["v"])


def _plain_rules(st):
    V = st["case"]["vocab"]
    tree, place, first, count = _places(st)
    seq = st["seqs"].long()[tree]
    l = st["logits"].float()
    if st["repetition"] is not None:
        pos = torch.arange(st["history"].shape[1], device="cuda")
        held = pos < st["lens"][:, None]
        counted = held & (pos >= st["counted_from"][:, None])
        zero = torch.zeros((st["lens"].numel(), V), dtype=torch.int32, device="cuda")
        seen = zero.scatter_add(1, st["history"].long(), held.int())[seq]
        n = zero.scatter_add(1, st["history"].long(), counted.int())[seq]
        if st["drafted"] is not None:   # the tokens of each row's own path
            parents = _padded_parents(st)
            at = (first[:, None] + torch.arange(st["widest"], device="cuda")).clamp(max=st["rows"] - 1)
            there = torch.arange(st["widest"], device="cuda") < count[:, None]
            above = (_ancestors(parents) & there[:, None, :])[tree, place].int()
            tokens = st["drafted"].long()[at][tree]
            seen, n = seen.scatter_add(1, tokens, above), n.scatter_add(1, tokens, above)
        r, p, f = (st[name][seq][:, None] for name in ("repetition", "presence", "frequency"))
        l = torch.where(seen > 0, torch.where(l > 0, l / r, l * r), l)
        l = l - (f * n + p * (n > 0))
    if st["bias"] is not None:
        starts, tokens, values = st["bias"]
        of = torch.searchsorted(starts.long(), torch.arange(tokens.numel(), device="cuda"), right=True) - 1
        dense = torch.zeros((st["lens"].numel(), V), device="cuda")
        dense[of, tokens.long()] = values
        l = l + dense[seq]
    if st["masks"] is not None:
        v = torch.arange(V, device="cuda")
        allowed = (st["masks"][:, v // 32] >> (v % 32) & 1) > 0
        rows = st["mask_rows"].long()
        l = torch.where((rows < 0)[:, None] | allowed[rows.clamp(min=0)], l, -math.inf)
    return l


def _frequencies(case):
    """Radians a position of each pair, in 64 bits."""
    sc, rot = _SCALING[case["scaling"]], case["rot"]
    base = 10000.0
    if sc.get("kind") == "base" and rot > 2:
        base *= sc["factor"] ** (rot / (rot - 2))
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if sc.get("kind") == "linear":
        f = f / sc["factor"]
    if sc.get("kind") == "bands":
        turns = sc["original_len"] * f / (2 * math.pi)   # over the length that the model was trained with
        keep = np.clip((turns - sc["low"]) / (sc["high"] - sc["low"]), 0.0, 1.0)
        f = f * (keep + (1 - keep) / sc["factor"])
    return f, sc.get("amplitude", 1.0)


def _plain_rope(st):
    case, rot = st["case"], st["case"]["rot"]
    f, amplitude = _frequencies(case)
    angle = st["positions"].double()[:, None] * torch.from_numpy(f).cuda()   # far positions: 64 bits
    c, s = ((amplitude * t(angle)).float()[:, None, :] for t in (torch.cos, torch.sin))
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        if case["half"]:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
        out[name] = torch.cat([y, x[..., rot:]], dim=-1).to(st[name].dtype)
    return out


# --------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    elt = _SIZES[case["dtype"]]
    if case["op"] == "rope":
        rows, heads = case["rows"], case["heads"] + case["kv"]
        return dict(bytes=2 * rows * heads * case["hs"] * elt + 4 * rows, flops=3 * rows * heads * case["rot"])
    a, nodes = _sizes(case)
    rows = int(nodes.sum())
    if case["op"] == "rules":
        V = case["vocab"]
        return dict(bytes=rows * V * (elt + 4) + (4 * int(a.sum()) if case["penalties"] else 0) + (4 * V if case["masks"] else 0),
                    flops=rows * V * (4 if case["penalties"] else 1))
    row = 2 * case["kv"] * case["hs"] * elt   # K and V of one position
    if case["op"] == "attn":
        qo = 2 * rows * case["heads"] * case["hs"] * elt
        seen = int((a * nodes).sum()) + rows * 2   # committed rows, and about two drafted ones
        return dict(bytes=int((a + nodes).sum()) * row + qo + 4 * int((-(-(a + nodes) // case["page"])).sum()),
                    flops=4 * case["heads"] * case["hs"] * seen)
    moved = sum(sum(1 for j, p in enumerate(path) if j != p) for path in prepare_paths(case))
    return dict(bytes=2 * moved * row * case["layers"] + 12 * rows + 4 * case["seqs"] * 4, flops=0)


def prepare_paths(case):
    """The accepted tokens of a seed's trees (how many there are hardly depends on the seed)."""
    rng = np.random.default_rng(1)
    _, nodes = _sizes(case)
    return [_accepted_tree(int(m), case["most"], rng)[1] for m in nodes]


# --------------------------------------------------------------------------
# the operators' definition, sequence by sequence

def exact(case, seed):
    st = prepare(case, seed)
    return {"attn": _exact_attention, "accept": _exact_accept, "rules": _exact_rules, "rope": _exact_rope}[case["op"]](st)


def _line(parents, i):
    """Token i and those above it."""
    got = []
    while i >= 0:
        got.append(i)
        i = int(parents[i])
    return got


def _exact_attention(st):
    case, p, ps = st["case"], st["host"], st["case"]["page"]
    H, KV, hs = case["heads"], case["kv"], case["hs"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    flat_k, flat_v = (t[0].transpose(1, 2).reshape(-1, KV, hs) for t in (st["k"], st["v"]))
    for i, s in enumerate(p["order"]):
        first, base = int(p["starts"][i]), int(p["prefix"][s])
        ids = [int(p["table"][s, t // ps]) * ps + t % ps for t in range(base + len(p["trees"][i]))]
        at = torch.tensor(ids, dtype=torch.long, device="cuda")
        k, v = flat_k[at].double(), flat_v[at].double()
        for u in range(len(p["trees"][i])):
            mine = list(range(base)) + sorted(base + a for a in _line(p["trees"][i], u))
            mine = torch.tensor(mine, dtype=torch.long, device="cuda")
            kk, vv = k[mine], v[mine]
            q = st["q"][first + u].double()
            kv_of = torch.tensor([h * KV // H for h in range(H)], device="cuda")
            x = torch.einsum("hd,thd->ht", q, kk[:, kv_of]) / math.sqrt(hs)
            out[first + u] = torch.einsum("ht,thd->hd", torch.softmax(x, dim=1), vv[:, kv_of])
    return out


def _exact_accept(st):
    case, p, ps = st["case"], st["host"], st["case"]["page"]
    refs, lens = p["refs"].copy(), (p["prefix"] + p["nodes"]).astype(np.int32)
    path = np.full(st["rows"], -1, np.int32)
    counts, following = [], []
    moves = []
    for i, s in enumerate(p["order"]):
        first, base, got = int(p["starts"][i]), int(p["prefix"][s]), p["paths"][i]
        path[first:first + len(got)] = got
        counts.append(len(got))
        following.append(int(p["targets"][first + got[-1]]))
        moves += [(s, base + a, base + j) for j, a in enumerate(got) if a != j]
        lens[s] = base + len(got)
        for c in range(-(-int(lens[s]) // ps), -(-(base + len(p["trees"][i])) // ps)):
            refs[p["table"][s, c]] -= 1
    if moves:
        where = lambda t: (torch.tensor([int(p["table"][m[0], m[t] // ps]) for m in moves], device="cuda"),  # noqa: E731
                           torch.tensor([m[t] % ps for m in moves], device="cuda"))
        (a, x), (b, y) = where(1), where(2)
        for pool in (st["k"], st["v"]):
            for layer in range(case["layers"]):
                for g in range(case["kv"]):
                    head = pool[layer, :, g]
                    head[b, y] = head[a, x].clone()
    dev = lambda z: torch.tensor(np.asarray(z), dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(path=dev(path), counts=dev(counts), next=dev(following), refs=dev(refs), lens=dev(lens), k=st["k"], v=st["v"])


def _exact_rules(st):
    p, V = st["host"], st["case"]["vocab"]
    out = st["logits"].double()
    history = st["history"].cpu().numpy()
    drafted = None if st["drafted"] is None else st["drafted"].cpu().numpy()
    for i, parents in enumerate(p["trees"]):
        first, n = int(p["starts"][i]), int(p["hist"][i])
        bias = None
        if st["bias"] is not None:
            starts, tokens, values = (t.cpu().numpy() for t in st["bias"])
            mine = slice(int(starts[i]), int(starts[i + 1]))
            bias = np.zeros(V)
            bias[tokens[mine]] = values[mine]
            bias = torch.from_numpy(bias).cuda()
        for u in range(len(parents)):
            l = out[first + u]
            if st["repetition"] is not None:
                extra = [] if drafted is None else [int(drafted[first + a]) for a in _line(parents, u)]
                seen = np.bincount(np.concatenate([history[i, :n], extra]).astype(np.int64), minlength=V)
                some = np.bincount(np.concatenate([history[i, n // 3:n], extra]).astype(np.int64), minlength=V)
                seen, some = torch.from_numpy(seen).cuda() > 0, torch.from_numpy(some).cuda().double()
                r, a, f = (float(st[name][i]) for name in ("repetition", "presence", "frequency"))
                l = torch.where(seen, torch.where(l > 0, l / r, l * r), l) - f * some - a * (some > 0)
            if bias is not None:
                l = l + bias
            if st["masks"] is not None and int(st["mask_rows"][first + u]) >= 0:
                words = st["masks"][int(st["mask_rows"][first + u])].cpu().numpy().view(np.uint8)
                bits = np.unpackbits(words, bitorder="little")[:V]
                l = torch.where(torch.from_numpy(bits).cuda() > 0, l, -math.inf)
            out[first + u] = l
    return out


def _exact_rope(st):
    case, rot = st["case"], st["case"]["rot"]
    f, amplitude = _frequencies(case)
    angle = st["positions"].double()[:, None] * torch.from_numpy(f).cuda()
    turn = torch.polar(torch.full_like(angle, amplitude), angle)   # amplitude * e^(i angle)
    out = {}
    for name in ("q", "k"):
        x = st[name].double()
        y = x.clone()
        first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if case["half"] else (slice(0, rot, 2), slice(1, rot, 2))
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out
