"""The paged cache on the GPU, call by call: what the documentation allows and other tests do not make.  Helpers and
tolerances are those of tests/test_gpu_pages.py."""
import math

import numpy as np
import pytest

from tests import pages_plan

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import llama_transformer_decode_gb300 as pkg  # noqa: E402,F401
from tests.test_gpu_pages import DT, check_wide, dev, wide_pool  # noqa: E402


def grouped(dtype, groups, lens, kv, hs, ps, seed, order="head"):
    """A pool whose sequences come in groups of (prefix, members) that share their prefix: whole pages by reference, the rest
    copied.  Returns the pool, the rows of a sequence in 64 bits, and the call's group arguments."""
    sizes, prefixes = [m for _, m in groups], [p for p, _ in groups]
    starts = np.concatenate([[0], np.cumsum(sizes)])
    firsts, prefix = np.repeat(starts[:-1], sizes), np.repeat(prefixes, sizes)
    pool, rows = wide_pool(dtype, len(firsts), kv, hs, ps, lens, [(int(f), int(p) // ps * ps) for f, p in zip(firsts, prefix)], seed=seed, order=order)
    for g, (p, m) in enumerate(groups):
        tail, a, b = p % ps, int(starts[g]), int(starts[g + 1])
        if tail and m > 1:
            pages = pool.table[a:b, p // ps].long()
            for t in (pool.k, pool.v):
                t[0, pages[1:], :, :tail] = t[0, pages[:1], :, :tail].expand(m - 1, -1, -1, -1)
    return pool, rows, dict(group_starts=dev(starts), prefix_lens=dev(prefixes))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(pages_plan.CROSSED)))
def test_blocks_that_go_on_to_another_item(case, dtype):
    """Blocks of the tensor-core role whose items leave the slots' tiles changed over (tests/test_attn_slots.py)."""
    groups, _, H, kv, hs = pages_plan.CROSSED[case]
    lens = pages_plan.crossed_lens(case)
    pool, rows, args = grouped(dtype, groups, lens, kv, hs, 64, seed=case)
    q = torch.randn((len(lens), H, hs), device="cuda").to(DT[dtype])
    lse = torch.empty((len(lens), H), device="cuda")
    out = pool.attention(q, 0, lse=lse, **args)
    pool.check()
    some = np.concatenate([[0], np.cumsum([m for _, m in groups])[:-1], [len(lens) - 1]])[:: max(1, len(groups) // 4)]
    check_wide(out, lse, q, rows, dtype, 1 / math.sqrt(hs), sorted({int(b) for b in some}))
    for _ in range(5):
        assert torch.equal(pool.attention(q, 0, **args), out)
    pool.check()
