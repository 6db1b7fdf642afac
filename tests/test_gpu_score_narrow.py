"""Alternatives of narrow rows, which leave some or most threads without elements.  Tolerances are test_gpu_score's."""
import math

import pytest

from test_gpu_score import check, make, scores, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("k", [1, 2, 3, 8, 9, 20, 64])
def test_narrow_rows(io, k):
    for vocab in (64, 65, 511, 512, 513, 540, 1791, 1792, 1793, 1800, 2000, 3583, 3584, 3592, 3600, 4096, 4100):
        x, t = make(7, vocab, io, seed=vocab)
        x[1, 1::2] = -math.inf                       # half of the entries masked, and all but a few
        x[2, 5:] = -math.inf
        x[3] = 0.5                                   # equal everywhere
        x[4, ::3] = torch.finfo(x.dtype).min
        t[1:4] = 0
        check(x, t, k, scores(x, t, k, io))
