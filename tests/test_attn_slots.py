"""The waits of the 16-bit tensor-core attention, on the CPU: the order in which a slot's issuing warp meets tiles
(csrc/attn_slots.h, the code the kernel runs) under the barriers' rules, with copies and products that end at any time
(tests/slot_order.cpp).  No wait passes before its tile is there, no stage is filled while it is read, everything ends."""
import itertools
import os
import subprocess

import pytest

from tests import pages_plan

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def simulate(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("slots") / "slot_order")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-pthread", "-I", pages_plan.CSRC,
                    os.path.join(HERE, "slot_order.cpp"), "-o", exe], check=True)

    def run(stages, seeds, lists):
        """lists: items as numbers of tiles, negative where both slots take every tile."""
        words = []
        for items in lists:
            words += (["0"] if words else []) + [str(n) for n in items]
        r = subprocess.run([exe, str(stages), str(seeds), *words], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout
        assert r.stdout.strip() == "ok"
    return run


# stages of a ring: head sizes up to 64, and above; and what neither uses
SHAPES = [4, 2, 3]


@pytest.mark.parametrize("stages", SHAPES)
def test_every_order_of_short_items(simulate, stages):
    kinds = [1, 2, 3, -1, -2]
    simulate(stages, 3, [x for n in (1, 2, 3) for x in itertools.product(kinds, repeat=n)])


@pytest.mark.parametrize("stages", SHAPES)
def test_items_of_many_tiles(simulate, stages):
    simulate(stages, 12, [(1, 51), (52, 1, 9), (7, -8, 5), (-5, 1, 1, 1, 12), (1,) * 12 + (20,), (3, -1, 3, -1, 3, -1, 10)])


@pytest.mark.parametrize("case", range(len(pages_plan.CROSSED)))
def test_blocks_of_planned_calls(simulate, case):
    groups, _, heads, kv, hs = pages_plan.CROSSED[case]
    stages = 2 if hs > 64 else 4
    blocks = pages_plan.tc_blocks(groups, pages_plan.crossed_lens(case), heads, kv, hs)
    crossed = [b for b in blocks if pages_plan.slots_change(b, stages)]
    assert crossed, "a call whose blocks do not cross slots tests nothing"
    simulate(stages, 4, [[-n if both else n for _, _, _, n, both in b] for b in crossed])


def test_the_replayed_plan_covers_every_tile_once():
    for case, (groups, _, heads, kv, hs) in enumerate(pages_plan.CROSSED):
        seen = {}
        for b in pages_plan.tc_blocks(groups, pages_plan.crossed_lens(case), heads, kv, hs):
            for g, item, k0, n, _ in b:
                for k in range(k0, k0 + n):
                    seen[g, item, k] = seen.get((g, item, k), 0) + 1
        assert seen and set(seen.values()) == {1}
        for g in {g for g, _, _ in seen}:
            tiles = {k for h, _, k in seen if h == g}
            items = {i for h, i, _ in seen if h == g}
            assert len([1 for h, _, _ in seen if h == g]) == len(items) * (max(tiles) + 1)
