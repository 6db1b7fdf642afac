"""bf16 rows are rounded once, from products of factors with two terms or more (rule_rounding): the scans of few, of
more and of many slices, and the gradients, against the 64-bit results rounded to bf16."""
import pytest
import torch

import rule_rounding as Q
from test_gpu_rule import backward, forward, make, many, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,hk,hv,dk,dv", [(2, 2, 4, 128, 128), (2, 1, 2, 64, 80), (2, 1, 2, 256, 96),
                                               (20, 4, 8, 128, 128), (70, 2, 4, 128, 128), (70, 2, 8, 64, 64)])
def test_one_rounding(batch, hk, hv, dk, dv):
    x = many(batch, hk, hv, dk, dv, io="bf16") if batch > 9 else make([200, 17], hk, hv, dk, dv, "bf16")
    want, parts, got = reference(x), Q.parts(x), {**forward(x), **backward(x)}
    for name in ("o", "dq", "dk", "dv"):
        assert got[name].dtype is torch.bfloat16
        assert Q.from_rounded(got[name], want[name]) <= Q.bound(name, parts), name
