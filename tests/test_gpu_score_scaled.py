"""Gradients of scaled losses: the entropy's part of a masked entry is 0 however large its gradient is.  Tolerances are
test_gpu_score's."""
import math

import pytest
import torch

from test_gpu_score import T, check_gradient, make, scores

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.0 ** 32, 1e20])
def test_masked_entries_with_a_large_gradient(io, scale):
    x, t = make(4, 2000, io)
    x[:, 1000:] = -math.inf
    x[:, 900:1000] = torch.finfo(x.dtype).min
    t %= 900
    fwd, out = scores(x, t, 0, io), torch.empty_like(x)
    given = dict(d_logp=torch.full((4,), scale, device="cuda"), d_entropy=torch.full((4,), -scale, device="cuda"),
                 entropy=fwd["entropy"])
    T.gdn_token_scores_backward(T.score_dims(4, 2000, 0, io), x, t, fwd["lse"], fwd["entropy"], given["d_logp"],
                                given["d_entropy"], out)
    check_gradient(x, t, out, given, io, fwd["lse"])
    assert (out[:, 900:] == 0).all()
