"""The plan of a paged attention call over 16-bit caches, replayed on the CPU: which blocks take the tensor-core role and the
items each of them works on.  Constants come from the kernel's sources."""
import os
import re

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "llama_transformer_decode_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


_H, _P, _L = _source("attn_pages.cuh"), _source("attn_plan.cuh"), _source("l2_pages.h")


def _number(text, name):
    m = re.search(r"\b%s = (\d+)\b" % name, text)
    assert m, name
    return int(m.group(1))


M, TC_ROWS = _number(_H, "kM"), _number(_H, "kTcRows")
TC_ITEM, ITEM, UNIT, LEAST16 = (_number(_H, n) for n in ("kTcItemCost", "kItemCost", "kCostUnit", "kTcLeast16"))
WARPS = _number(_L, "kWalkWarps")
_c = re.search(r"return n > kTcRows \? \(hs > 64 \? (\d+) : (\d+)\) : \(hs > 64 \? (\d+) : (\d+)\);", _H)
_s = re.search(r"int attn_pages_16_shift\(int hs\) \{ return hs <= 64 \? (\d+) : (\d+); \}", _source("attn_pages_16.cu"))
assert _c and _s
KEYS, RUN = 128, 2 * TC_ROWS


def cdiv(a, b):
    return -(-a // b)


def tc_cost(n, hs):
    big, small = (_c.group(1), _c.group(2)), (_c.group(3), _c.group(4))
    return int((big if n > TC_ROWS else small)[0 if hs > 64 else 1])


def tc_blocks(groups, lens, heads, kv, hs, sms=152):
    """groups: (prefix, rows); lens: every row's length.  Per tensor-core block its segments (group, item, first tile, tiles, both slots)."""
    gq = cdiv(heads, kv)
    shift = int(_s.group(1 if hs <= 64 else 2))
    starts = np.concatenate([[0], np.cumsum([r for _, r in groups])])
    minlen = [0 if r < 2 else min([p] + [int(n) for n in lens[starts[g]:starts[g] + r]]) for g, (p, r) in enumerate(groups)]
    full = []
    for (_, r), m in zip(groups, minlen):
        n, keys = r * gq, m // KEYS * KEYS
        worth = n > M and cdiv(n, M) * kv * len(groups) * UNIT * (keys >> shift) >= LEAST16
        full.append(keys // KEYS if worth else 0)
    t0, at = [], 0
    for (_, r), f in zip(groups, full):
        t0.append(at)
        at += (TC_ITEM + f * tc_cost(r * gq, hs)) * cdiv(r * gq, RUN) * kv if f else 0
    tc = at
    cost = 0
    for (_, r), m, f in zip(groups, minlen, full):
        kt = cdiv(m - f * KEYS, 1 << shift)
        cost += cdiv(r * gq, M) * kv * (ITEM + kt * UNIT) if kt else 0
    for g, (_, r) in enumerate(groups):
        for n in lens[starts[g]:starts[g] + r]:
            kt = cdiv(int(n) - minlen[g], 1 << shift)
            cost += cdiv(gq, M) * kv * (ITEM + kt * UNIT) if kt else 0
    if not tc:
        return []
    t, w = np.float32(tc), np.float32(cost)
    most = sms - (1 if cost else 0)
    n_tc = max(1, min(int(np.float32(sms) * (t / (t + w))), most))

    def slower(n):
        return max(t / np.float32(n), w / np.float32(sms - n) if cost else np.float32(0))
    if n_tc < most and slower(n_tc + 1) < slower(n_tc):
        n_tc += 1
    per = max(TC_ITEM + tc_cost(2 * TC_ROWS, hs), cdiv(tc, n_tc))
    blocks = []
    for b in range(cdiv(tc, per)):
        x, x_end, segs = b * per, min((b + 1) * per, tc), []
        for g, (_, r) in enumerate(groups):
            if not full[g]:
                continue
            n, c = r * gq, tc_cost(r * gq, hs)
            length = TC_ITEM + full[g] * c
            for item in range(cdiv(n, RUN) * kv):
                lo = t0[g] + item * length
                places = [lo if k == 0 else lo + TC_ITEM + k * c for k in range(full[g])] if lo < x_end and lo + length > x else []
                mine = [k for k, p in enumerate(places) if x <= p < x_end]
                if mine:
                    rows = min(RUN, n - item % cdiv(n, RUN) * RUN)
                    segs.append((g, item, mine[0], len(mine), rows > TC_ROWS))
        blocks.append(segs)
    return blocks


def slots_change(segs, stages):
    """Whether some stage's last tile, when a block comes to use it again, was one that a slot which takes the new tile did not take."""
    takers = {}
    t = 0
    for _, _, _, n, both in segs:
        for i in range(n):
            now = {0, 1} if both else {i & 1}
            if (t + i) % stages in takers and not now <= takers[(t + i) % stages]:
                return True
            takers[(t + i) % stages] = now
        t += n
    return False


# Calls whose plan has blocks that go on from one item to another with the slots' tiles changed over, or from an item of one
# tile: groups of (prefix, rows), most own rows, heads, KV heads, head size.
CROSSED = [
    ([(16384, 64)], 512, 32, 32, 128),
    ([(4000, 24)], 30, 32, 8, 128),
    ([(130, 40)] * 12 + [(1500, 40)], 3, 32, 16, 128),
    ([(3662, 34), (1011, 22), (2459, 6), (1096, 45), (819, 39), (433, 22), (1185, 44), (2536, 32)], 4, 64, 8, 96),
    ([(966, 27), (456, 6), (1336, 29), (710, 39), (3210, 30), (983, 11)], 4, 16, 4, 128),
    ([(1146, 33), (882, 20), (748, 36), (530, 16), (898, 44), (3219, 19), (400, 17), (668, 18)], 4, 64, 8, 64),
    ([(1071, 12), (166, 42), (1176, 40), (547, 12), (397, 40), (3513, 18), (859, 4)], 4, 16, 8, 64),
    ([(682, 48), (2658, 41), (478, 13), (1730, 46), (585, 27), (287, 46), (1000, 37), (665, 3)], 4, 64, 8, 48),
]


def crossed_lens(case):
    groups, own = CROSSED[case][:2]
    prefix = np.repeat([p for p, _ in groups], [r for _, r in groups])
    return prefix + np.random.default_rng(case).integers(0, own + 1, len(prefix))
