"""How a paged attention call's blocks divide into the walk and the tensor-core role (csrc/attn_split.h, the code the plan runs),
compiled for the CPU with every division by zero and signed overflow a trap."""
import os
import subprocess

import numpy as np
import pytest

from tests import pages_plan

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("split") / "role_split")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fsanitize=integer-divide-by-zero,signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", pages_plan.CSRC, os.path.join(HERE, "role_split.cpp"), "-o", exe], check=True)

    def run(calls):
        r = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in calls), capture_output=True, text=True)
        assert r.returncode == 0, r
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


@pytest.mark.parametrize("blocks", [152, 148, 2])
def test_every_tile_has_a_taker_and_no_role_without_work_blocks(split, blocks):
    rng = np.random.default_rng(blocks)
    sizes = [0, 1, 7, 40, 90, 1000, 36_257, 2_000_000, 900_000_000]
    calls = [(w, t, blocks, 8, lw, lt) for w in sizes + rng.integers(1, 1 << 30, 40).tolist() for t in sizes + rng.integers(1, 1 << 30, 40).tolist()
             for lw, lt in ((11, 112), (400, 170))]
    for (walk, tc, _, warps, least_walk, least_tc), (n_tc, per_tc, per) in zip(calls, split(calls)):
        assert 0 <= n_tc <= blocks and per >= least_walk
        if tc:
            assert n_tc >= 1 and per_tc >= least_tc and n_tc * per_tc >= tc > (n_tc - 1) * per_tc
        else:
            assert n_tc == 0
        if walk:
            assert n_tc < blocks and per * (blocks - n_tc) * warps >= walk


def test_a_call_whose_keys_all_lie_in_whole_tensor_core_tiles(split):
    """The walk has no cost and every block the other role: attention right after a long prompt was forked."""
    (n_tc, per_tc, per), = split([(0, 8 * (80 + 128 * 38), 152, 8, 11, 118)])
    assert n_tc == 152 and per == 11 and per_tc * 152 >= 8 * (80 + 128 * 38)
