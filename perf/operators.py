"""Measured cases of the paged-cache operators: appending rows, forking,
freeing and compacting sequences of a page pool, and the decode attention of a
batch whose sequences share long prefixes.

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, through the package's ``PagePool``.

A pool holds K and V as [layer][page][kv head][row][head size], a reference
count per page, and per sequence its length and its page table.  Sequences of
``prepare`` hold pages in shuffled order, as in a pool that has served for a
while.  The operators that change the bookkeeping (counts, lengths, tables)
start every pass from the same bookkeeping, copied from a kept original; the
rows they move are then the same in every pass.
"""
import math
import zlib

import numpy as np
import torch

own = False

_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------
# cases

def listed():
    return [
        # a small model's step: four sequences, a short system prompt (latency of one call)
        dict(name="attn_tiny_fp32", op="attn", dtype="fp32", heads=8, kv=4, hs=8, page=16, groups="4",
             prefix="100", suffix_lo=1, suffix_hi=20),
        # a mid-size model, 16 chats under one system prompt, cache in bf16
        dict(name="attn_mid_bf16", op="attn", dtype="bf16", heads=12, kv=12, hs=64, page=16, groups="16",
             prefix="515", suffix_lo=1, suffix_hi=300),
        # grouped heads, fp32 cache as the decoder keeps it, 64 sequences on one 1000-token prompt
        dict(name="attn_gqa_fp32", op="attn", dtype="fp32", heads=32, kv=4, hs=64, page=64, groups="64",
             prefix="1001", suffix_lo=16, suffix_hi=1000),
        # the 7B head shape, fp32 cache, long documents
        dict(name="attn_7b_fp32", op="attn", dtype="fp32", heads=32, kv=32, hs=128, page=32, groups="32",
             prefix="2048", suffix_lo=100, suffix_hi=1500),
        # grouped heads in fp16, several prefixes of odd lengths in one batch, one sequence without a prefix
        dict(name="attn_gqa_fp16_groups", op="attn", dtype="fp16", heads=32, kv=4, hs=64, page=32, groups="30,1,17,12,4",
             prefix="16390,0,4099,33,8190", suffix_lo=1, suffix_hi=700),
        # the 7B head shape in bf16: 64 questions to one 16k-token document
        dict(name="attn_7b_bf16_long", op="attn", dtype="bf16", heads=32, kv=32, hs=128, page=64, groups="64",
             prefix="16384", suffix_lo=1, suffix_hi=512),
        # one layer's rows of a decode step of 64 sequences
        dict(name="append_step_bf16", op="append", dtype="bf16", layers=22, layer=0, kv=4, hs=64, page=16, seqs=64,
             len_lo=1, len_hi=600, new_lo=1, new_hi=1),
        # prompts of ragged lengths brought in for every layer at once
        dict(name="append_prompts_fp32", op="append", dtype="fp32", layers=12, layer=-1, kv=12, hs=64, page=32, seqs=24,
             len_lo=0, len_hi=200, new_lo=1, new_hi=700),
        # four continuations of one sequence of a small model
        dict(name="fork_tiny_fp32", op="fork", dtype="fp32", layers=5, kv=4, hs=8, page=16, parents=1, children=4,
             len_lo=70, len_hi=70),
        # a prompt of the 7B shape forked into 63 sequences: the last page is copied for each
        dict(name="fork_7b_bf16", op="fork", dtype="bf16", layers=32, kv=32, hs=128, page=16, parents=1, children=63,
             len_lo=1033, len_hi=1033),
        # 16 finished sequences given back
        dict(name="free_bf16", op="free", dtype="bf16", layers=12, kv=12, hs=64, page=16, seqs=64, gone=16, compact=False,
             len_lo=50, len_hi=900),
        # half of the sequences given back and the pool closed up
        dict(name="free_compact_fp32", op="free", dtype="fp32", layers=22, kv=4, hs=64, page=32, seqs=64, gone=31,
             compact=True, len_lo=16, len_hi=900),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# (query heads, KV heads, head size): the decoder's shapes
_HEADS = [(8, 4, 8), (6, 4, 48), (12, 12, 64), (32, 4, 64), (32, 32, 128), (32, 8, 128), (16, 2, 64), (8, 1, 128)]


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "fork", "free"])
    dtype = rng.choice(["fp32", "bf16", "fp16"])
    heads, kv, hs = rng.choice(_HEADS)
    page = rng.choice([16, 32, 64, 128])
    if op == "attn":
        n_groups = rng.choice([1, 1, 1, 2, 3, 5])
        sizes = [_log_int(rng, 1, 64 // n_groups) for _ in range(n_groups)]
        top = 12000 if kv * hs >= 4096 and n_groups == 1 else 6000
        if kv * hs >= 1024 and dtype == "fp32":
            top = 3000
        prefix = [_log_int(rng, 16, top) for _ in sizes]
        hi = _log_int(rng, 4, 500 if kv * hs >= 1024 else 1000)
        return dict(op=op, dtype=dtype, heads=heads, kv=kv, hs=hs, page=page, groups=",".join(map(str, sizes)),
                    prefix=",".join(map(str, prefix)), suffix_lo=1, suffix_hi=hi)
    # whole pools are moved and compared: about 1.5 GB at most
    elt = 4 if dtype == "fp32" else 2
    layers = rng.randint(2, 32)
    rows_cap = int(1.5e9 / (2 * layers * kv * hs * elt))
    if op == "append":
        seqs = _log_int(rng, 1, 64)
        most = max(2, min(600, rows_cap // seqs - 2 * page))
        one = rng.random() < 0.5
        return dict(op=op, dtype=dtype, layers=layers, layer=rng.choice([-1, 0]), kv=kv, hs=hs, page=page, seqs=seqs,
                    len_lo=0, len_hi=most // 2, new_lo=1, new_hi=1 if one else _log_int(rng, 1, max(1, most // 2)))
    if op == "fork":
        parents = rng.randint(1, 4)
        length = _log_int(rng, 1, max(16, min(2000, (rows_cap - 64 * page) // parents)))
        room = max(1, (rows_cap - parents * (length + page)) // page // parents)
        return dict(op=op, dtype=dtype, layers=layers, kv=kv, hs=hs, page=page, parents=parents,
                    children=_log_int(rng, 1, min(room, 64 // parents)), len_lo=max(1, length // 2), len_hi=length)
    seqs = rng.randint(2, 64)
    most = max(2, min(900, rows_cap // seqs - 2 * page))
    return dict(op=op, dtype=dtype, layers=layers, kv=kv, hs=hs, page=page, seqs=seqs, gone=rng.randint(1, seqs - 1),
                compact=rng.random() < 0.7, len_lo=1, len_hi=most)


def _ints(text):
    return [int(t) for t in text.split(",")]


# --------------------------------------------------------------------------
# inputs

def _plan(case, seed):
    """Bookkeeping of a pool on the host: counts, lengths, tables, and the call's index arrays.  The lengths are the
    case's (so that its shapes are); which pages and sequences, and in what order, is the seed's."""
    sizes_of = np.random.default_rng(zlib.crc32(repr(sorted((a, b) for a, b in case.items() if a != "name")).encode()))
    rng = np.random.default_rng(seed)
    ps = case["page"]
    up = lambda n: -(-n // ps)  # noqa: E731
    op = case["op"]
    extra = {}
    if op == "attn":
        sizes, prefix = _ints(case["groups"]), _ints(case["prefix"])
        lens, first = [], []
        for n, p in zip(sizes, prefix):
            first += [len(lens)] * n
            lens += [p + int(v) for v in sizes_of.integers(case["suffix_lo"], case["suffix_hi"] + 1, n)]
        shared = [prefix[g] // ps for g, n in enumerate(sizes) for _ in range(n)]
        need = sum(up(n) for n in lens) - sum((n - 1) * (q // ps) for n, q in zip(sizes, prefix))
        extra = dict(starts=np.concatenate([[0], np.cumsum(sizes)]), prefix=np.array(prefix))
        n_seqs = len(lens)
    else:
        if op == "append":
            n = case["seqs"]
            lens = [int(v) for v in sizes_of.integers(case["len_lo"], case["len_hi"] + 1, n)]
            new = sizes_of.integers(case["new_lo"], case["new_hi"] + 1, n)
            need = sum(up(a + int(b)) for a, b in zip(lens, new))
            n_seqs = n
            order = rng.permutation(n)
            extra = dict(seqs=order, starts=np.concatenate([[0], np.cumsum(new[order])]))
        elif op == "fork":
            n, c = case["parents"], case["children"]
            lens = [int(v) for v in sizes_of.integers(case["len_lo"], case["len_hi"] + 1, n)] + [0] * (n * c)
            need = sum(up(v) for v in lens) + n * c
            n_seqs = n + n * c
            extra = dict(src=np.repeat(np.arange(n), c), dst=n + rng.permutation(n * c))
        else:
            n_seqs = case["seqs"]
            lens = [int(v) for v in sizes_of.integers(case["len_lo"], case["len_hi"] + 1, n_seqs)]
            need = sum(up(v) for v in lens)
            extra = dict(seqs=rng.permutation(n_seqs)[:case["gone"]])
        first, shared = list(range(n_seqs)), [0] * n_seqs
    n_pages = need + 3
    reach = max(lens) + (int((extra["starts"][1:] - extra["starts"][:-1]).max()) if op == "append" else 0)
    max_pages = up(reach) + 1
    table = np.full((n_seqs, max_pages), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    ids = rng.permutation(n_pages)
    nxt = 0
    for s, length in enumerate(lens):
        for i in range(up(length)):
            if first[s] != s and i < shared[s]:
                table[s, i] = table[first[s], i]
            else:
                table[s, i] = ids[nxt]
                nxt += 1
            refs[table[s, i]] += 1
    return dict(n_seqs=n_seqs, n_pages=n_pages, max_pages=max_pages, lens=lens, first=first, table=table, refs=refs, **extra)


def prepare(case, seed):
    p = _plan(case, seed)
    dt = _DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dt)

    layers = case.get("layers", 1)
    shape = (p["n_pages"], case["kv"], case["page"], case["hs"])
    k, v = (torch.empty((layers, *shape), dtype=dt, device="cuda") for _ in range(2))
    for t in (k, v):
        for i in range(layers):
            t[i] = normal(*shape)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    # one block of integers: counts, lengths, tables (so a pass can start from the same bookkeeping)
    book0 = dev(np.concatenate([p["refs"], np.array(p["lens"]), p["table"].ravel()]))
    book = book0.clone()
    a, b = p["n_pages"], p["n_pages"] + p["n_seqs"]
    st = dict(case=case, k=k, v=v, book0=book0, book=book, refs=book[:a], lens=book[a:b],
              table=book[b:].view(p["n_seqs"], p["max_pages"]), host=p)
    op = case["op"]
    if op == "attn":
        # queries that concentrate on some keys, as trained heads do
        st["q"] = normal(p["n_seqs"], case["heads"], case["hs"], std=2.0)
        st["starts"], st["prefix"] = dev(p["starts"]), dev(p["prefix"])
    elif op == "append":
        rows = int(p["starts"][-1])
        lead = (layers,) if case["layer"] < 0 else ()
        st["new_k"], st["new_v"] = normal(*lead, rows, case["kv"], case["hs"]), normal(*lead, rows, case["kv"], case["hs"])
        st["seqs"], st["starts"] = dev(p["seqs"]), dev(p["starts"])
        st["one"] = bool((np.diff(p["starts"]) == 1).all())
    elif op == "fork":
        st["src"], st["dst"] = dev(p["src"]), dev(p["dst"])
    else:
        st["seqs"] = dev(p["seqs"])
    if own:
        import llama_transformer_decode_gb300 as pkg
        st["pool"] = pkg.PagePool.from_tensors(k, v, refs=st["refs"], lens=st["lens"], table=st["table"])
    return st


# --------------------------------------------------------------------------
# one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _pool_out(st):
    out = dict(refs=st["refs"], lens=st["lens"], table=st["table"])
    if st["case"]["op"] != "free" or st["case"]["compact"]:   # freeing alone moves no rows
        out.update(k=st["k"], v=st["v"])
    return out


def _run_own(st):
    case, pool = st["case"], st["pool"]
    op = case["op"]
    if op == "attn":
        return pool.attention(st["q"], 0, group_starts=st["starts"], prefix_lens=st["prefix"])
    st["book"].copy_(st["book0"])
    if op == "append":
        pool.append(st["new_k"], st["new_v"], st["seqs"], starts=None if st["one"] else st["starts"],
                    layer=None if case["layer"] < 0 else case["layer"])
    elif op == "fork":
        pool.fork(st["src"], st["dst"])
    else:
        pool.free(st["seqs"], compact=case["compact"])
    return _pool_out(st)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "attn":
        return _plain_attention(st)
    st["book"].copy_(st["book0"])
    {"append": _plain_append, "fork": _plain_fork, "free": _plain_free}[op](st)
    return _pool_out(st)


def _plain_attention(st):
    case, host, ps = st["case"], st["host"], st["case"]["page"]
    H, KV, hs = case["heads"], case["kv"], case["hs"]
    q, out = st["q"].float(), torch.empty_like(st["q"])
    heads = torch.tensor([h * KV // H for h in range(H)], device="cuda")
    prefix = [int(host["prefix"][g]) for g in range(len(host["prefix"]))
              for _ in range(int(host["starts"][g + 1] - host["starts"][g]))]
    for b, n in enumerate(host["lens"]):
        pos = torch.arange(n, device="cuda")
        row = torch.where(pos < prefix[b], host["first"][b], b)
        page = st["table"][row, pos // ps]
        k = st["k"][0][page, :, pos % ps].float()   # [n][kv][hs]
        v = st["v"][0][page, :, pos % ps].float()
        if KV != H:
            k, v = k[:, heads], v[:, heads]
        s = torch.matmul(k.transpose(0, 1), q[b].unsqueeze(2)).squeeze(2) / math.sqrt(hs)  # [H][n]
        w = torch.exp(s - s.max(dim=1, keepdim=True).values)
        o = torch.matmul(w.unsqueeze(1), v.transpose(0, 1)).squeeze(1) / w.sum(dim=1, keepdim=True)
        out[b] = o.to(out.dtype)
    return out


def _lowest_free(refs):
    """Page ids, the free ones first and ascending."""
    return torch.sort((refs > 0).int(), stable=True).indices


def _plain_append(st):
    case, ps = st["case"], st["case"]["page"]
    refs, lens, table = st["refs"], st["lens"], st["table"]
    seqs, starts = st["seqs"].long(), st["starts"].long()
    total = st["new_k"].shape[-3]
    new = starts[1:] - starts[:-1]
    old = lens[seqs].long()
    have, want = (old + ps - 1) // ps, (old + new + ps - 1) // ps
    base = torch.cumsum(want - have, 0) - (want - have)      # pages taken by the sequences before
    free = _lowest_free(refs)
    cols = torch.arange(table.shape[1], device="cuda")[None]
    fresh = (cols >= have[:, None]) & (cols < want[:, None])
    ids = free[(base[:, None] + cols - have[:, None]).clamp(0, free.numel() - 1)]
    table[seqs] = torch.where(fresh, ids.int(), table[seqs])
    refs.index_add_(0, ids.reshape(-1), fresh.reshape(-1).int())
    lens[seqs] = (old + new).int()
    r = torch.arange(total, device="cuda")
    i = torch.searchsorted(starts, r, right=True) - 1
    pos = old[i] + r - starts[i]
    page, row = table[seqs[i], pos // ps].long(), pos % ps
    if case["layer"] < 0:
        st["k"].permute(1, 3, 0, 2, 4)[page, row] = st["new_k"].transpose(0, 1)
        st["v"].permute(1, 3, 0, 2, 4)[page, row] = st["new_v"].transpose(0, 1)
    else:
        st["k"][case["layer"]].permute(0, 2, 1, 3)[page, row] = st["new_k"]
        st["v"][case["layer"]].permute(0, 2, 1, 3)[page, row] = st["new_v"]


def _plain_fork(st):
    ps = st["case"]["page"]
    refs, lens, table = st["refs"], st["lens"], st["table"]
    src, dst = st["src"].long(), st["dst"].long()
    n = lens[src].long()
    full, tail = n // ps, n % ps
    cols = torch.arange(table.shape[1], device="cuda")[None]
    part = (tail > 0).long()
    ids = _lowest_free(refs)[torch.cumsum(part, 0) - part]
    keep = cols < full[:, None]
    rows = torch.where(keep, table[src], table[dst])
    rows = torch.where((cols == full[:, None]) & (part[:, None] > 0), ids[:, None].int(), rows)
    refs.index_add_(0, torch.where(keep, rows, 0).reshape(-1).long(), keep.reshape(-1).int())
    refs.index_add_(0, ids, part.int())
    old = table[src, full].long()                            # the page to copy from, where there is a tail
    table[dst] = rows
    lens[dst] = n.int()
    mask = (torch.arange(ps, device="cuda")[None] < tail[:, None])[None, :, None, :, None]
    for pool in (st["k"], st["v"]):
        from_ = torch.where(part > 0, old, ids)
        pool[:, ids] = torch.where(mask, pool[:, from_], pool[:, ids])


def _plain_free(st):
    case, ps = st["case"], st["case"]["page"]
    refs, lens, table = st["refs"], st["lens"], st["table"]
    seqs = st["seqs"].long()
    cols = torch.arange(table.shape[1], device="cuda")[None]
    held = cols < ((lens[seqs] + ps - 1) // ps)[:, None]
    refs.index_add_(0, torch.where(held, table[seqs], 0).reshape(-1).long(), -held.reshape(-1).int())
    lens[seqs] = 0
    if not case["compact"]:
        return
    live = refs > 0
    n_live = live.sum()
    ids = torch.arange(refs.numel(), device="cuda")
    moved = torch.nonzero(live & (ids >= n_live)).squeeze(1)
    holes = torch.nonzero(~live & (ids < n_live)).squeeze(1)
    to = ids.clone()
    to[moved] = holes
    st["k"][:, holes] = st["k"][:, moved]
    st["v"][:, holes] = st["v"][:, moved]
    refs[holes] = refs[moved]
    refs[moved] = 0
    held = cols < ((lens + ps - 1) // ps)[:, None]
    table.copy_(torch.where(held, to[torch.where(held, table, 0).long()].int(), table))


# --------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    p = _plan(case, 0)
    elt = 4 if case["dtype"] == "fp32" else 2
    ps, row = case["page"], 2 * case["kv"] * case["hs"] * elt   # K and V of one position
    up = lambda n: -(-n // ps)  # noqa: E731
    lens = p["lens"]
    op = case["op"]
    if op == "attn":
        sizes, prefix = _ints(case["groups"]), _ints(case["prefix"])
        own_rows = sum(lens) - sum(n * q for n, q in zip(sizes, prefix))
        keys = sum(prefix) + own_rows
        qo = 2 * p["n_seqs"] * case["heads"] * case["hs"] * elt
        return dict(bytes=keys * row + qo + 4 * -(-keys // ps), flops=4 * case["heads"] * case["hs"] * sum(lens))
    if op == "append":
        rows = int(p["starts"][-1]) * (case["layers"] if case["layer"] < 0 else 1)
        return dict(bytes=2 * rows * row + 8 * p["n_seqs"], flops=0)
    if op == "fork":
        c = case["children"]
        tails = sum(n % ps for n in lens)
        table = sum(up(n) for n in lens)
        return dict(bytes=case["layers"] * row * tails * (1 + c) + 4 * table * (1 + 3 * c), flops=0)
    held = sum(up(lens[s]) for s in p["seqs"])
    if not case["compact"]:
        return dict(bytes=4 * (3 * held + 2 * len(p["seqs"])), flops=0)
    refs = p["refs"].copy()
    for s in p["seqs"]:
        refs[p["table"][s, :up(lens[s])]] -= 1
    n_live = int((refs > 0).sum())
    moved = int((refs[n_live:] > 0).sum())
    return dict(bytes=case["layers"] * row * ps * moved * 2 + 4 * (2 * refs.size + 3 * held + 2 * n_live), flops=0)


# --------------------------------------------------------------------------
# the operators' definition, sequence by sequence

def exact(case, seed):
    st = prepare(case, seed)
    p, ps, op = st["host"], case["page"], case["op"]
    if op == "attn":
        return _exact_attention(st)
    refs, lens, table = p["refs"].copy(), np.array(p["lens"], np.int32), p["table"].copy()
    k, v = st["k"], st["v"]

    def take():
        i = int(np.flatnonzero(refs == 0)[0])
        refs[i] = 1
        return i

    if op == "append":
        layers = range(case["layers"]) if case["layer"] < 0 else [case["layer"]]
        todo = []
        for i, s in enumerate(p["seqs"]):
            for r in range(int(p["starts"][i]), int(p["starts"][i + 1])):
                n = int(lens[s])
                if n % ps == 0:
                    table[s, n // ps] = take()
                todo.append((int(table[s, n // ps]), n % ps))
                lens[s] += 1
        pages = torch.tensor([t[0] for t in todo], device="cuda")
        rows = torch.tensor([t[1] for t in todo], device="cuda")
        for layer in layers:
            nk, nv = (st["new_k"][layer], st["new_v"][layer]) if case["layer"] < 0 else (st["new_k"], st["new_v"])
            for g in range(case["kv"]):
                k[layer, :, g][pages, rows] = nk[:, g]
                v[layer, :, g][pages, rows] = nv[:, g]
    elif op == "fork":
        for s, d in zip(p["src"], p["dst"]):
            n = int(lens[s])
            for i in range(n // ps):
                table[d, i] = table[s, i]
                refs[table[s, i]] += 1
            if n % ps:
                i = n // ps
                table[d, i] = take()
                a, b = int(table[s, i]), int(table[d, i])
                k[:, b, :, :n % ps] = k[:, a, :, :n % ps]
                v[:, b, :, :n % ps] = v[:, a, :, :n % ps]
            lens[d] = n
    else:
        for s in p["seqs"]:
            for i in range(-(-int(lens[s]) // ps)):
                refs[table[s, i]] -= 1
            lens[s] = 0
        if case["compact"]:
            n_live = int((refs > 0).sum())
            holes = [i for i in range(n_live) if refs[i] == 0]
            moved = [i for i in range(n_live, refs.size) if refs[i] > 0]
            to = dict(zip(moved, holes))
            for a, b in to.items():
                k[:, b], v[:, b] = k[:, a].clone(), v[:, a].clone()
                refs[b], refs[a] = refs[a], 0
            for s in range(p["n_seqs"]):
                for i in range(-(-int(lens[s]) // ps)):
                    table[s, i] = to.get(int(table[s, i]), int(table[s, i]))
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    out = dict(refs=dev(refs), lens=dev(lens), table=dev(table))
    if op != "free" or case["compact"]:
        out.update(k=k, v=v)
    return out


def _exact_attention(st):
    case, p, ps = st["case"], st["host"], st["case"]["page"]
    H, KV, hs = case["heads"], case["kv"], case["hs"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for g in range(len(p["prefix"])):
        lo, hi = int(p["starts"][g]), int(p["starts"][g + 1])
        n0 = int(p["prefix"][g])

        def rows(pool, seq, a, b):
            ids = [int(p["table"][seq, t // ps]) * ps + t % ps for t in range(a, b)]
            flat = pool[0].transpose(1, 2).reshape(-1, KV, hs)
            return flat[torch.tensor(ids, dtype=torch.long, device="cuda")].double()

        k0, v0 = rows(st["k"], lo, 0, n0), rows(st["v"], lo, 0, n0)
        for b in range(lo, hi):
            n = int(p["lens"][b])
            k = torch.cat([k0, rows(st["k"], b, n0, n)])
            v = torch.cat([v0, rows(st["v"], b, n0, n)])
            for h0 in range(KV):
                hq = [h for h in range(H) if (h * KV) // H == h0]
                s = k[:, h0] @ st["q"][b, hq].double().T / math.sqrt(hs)   # [n][heads]
                out[b, hq] = torch.softmax(s, dim=0).T @ v[:, h0]
    return out
