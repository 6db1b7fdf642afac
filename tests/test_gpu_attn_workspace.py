"""One workspace for calls of different sizes: each gives the bits that it gives on a workspace of its own,
and leaves every arrival counter at zero."""
import os
import re

import pytest
import torch

from test_gpu_attn_verify import Case

pytestmark = pytest.mark.gpu
T = pytest.importorskip("tree_masked_gated_amd")

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_masked_gated_amd", "csrc",
                      "attn_verify.hpp")
COUNTERS = int(re.search(r"kCounterBytes = (\d+);", open(SOURCE).read()).group(1))


def cut_and_clean(ws):
    """Whether a block of rows was cut (partial results are there), and whether the counters are zero."""
    assert COUNTERS % 4 == 0 and ws.numel() > COUNTERS
    return bool(ws[COUNTERS:].any()), not bool(ws[:COUNTERS].any())


CASES = [
    ("tokens, 8 key heads", dict(sizes=[1] * 64, ctx=[700 + 9 * i for i in range(64)], kind="star", hq=16, hkv=8, d=128)),
    ("a part of them", dict(sizes=[1] * 8, ctx=[300 + 77 * i for i in range(8)], kind="star", hq=16, hkv=8, d=128)),
    ("one token, many parts", dict(sizes=[1], ctx=[40000], kind="star", hq=8, hkv=1, d=64)),
    ("trees of 20 rows", dict(sizes=[20] * 3, ctx=[2000, 10, 777], kind="rrt", hq=2, hkv=2, d=64)),
    ("blocks of 128 rows", dict(sizes=[25] * 33, ctx=[900 - 27 * i for i in range(33)], kind="rrt", hq=16, hkv=4, d=64)),
    ("blocks of 256 rows", dict(sizes=[40] * 33, ctx=[900 - 27 * i for i in range(33)], kind="rrt", hq=16, hkv=4, d=64)),
    ("blocks side by side", dict(sizes=[130] * 3, ctx=[1000, 37, 511], kind="rrt", hq=8, hkv=4, d=64)),
    ("ragged", dict(sizes=[9, 0, 40], ctx=[1300, 70, 2100], kind="rrt", hq=8, hkv=2, d=128, ragged=True)),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_one_workspace_for_calls_of_all_sizes(io):
    cases = []
    for i, (name, kw) in enumerate(CASES):
        print("[gpu-attn-workspace]", io, name, flush=True)
        c = Case(**kw, io=io, page=16, seed=i)
        o = c.call()
        cut, clean = cut_and_clean(c.ws)
        assert cut and clean, name
        c.check(o)
        cases.append((name, c, o))
    shared = torch.zeros(max(c.ws.numel() for _, c, _ in cases), dtype=torch.uint8, device="cuda")
    for _, c, _ in cases:
        c.ws = shared
    order = list(range(len(cases))) + list(range(len(cases)))[::-1] + [0, 1, 0, 5, 1, 5, 2, 0, 2]
    for i in order:
        name, c, want = cases[i]
        print("[gpu-attn-workspace]", io, name, flush=True)
        assert torch.equal(c.call().view(torch.uint8), want.view(torch.uint8)), (name, order)
        assert cut_and_clean(shared)[1], name
