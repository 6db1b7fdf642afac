"""Gradients of rows of logits far from 0, whose lse says little or nothing of ln s once it is rounded: rows that
hold nothing but a mask's value, and logits with a large common part.  Against 64 bits, from the logits less their
maximum; the tolerances are test_gpu_score's (the rounding of ln s, 2^-21, is within their 32 steps of 2^-24).
Nearer rows, |lse| below 4096, are formed from the lse that is given."""
import math

import pytest
import torch

from test_gpu_score import T, check_gradient, make, scores

pytestmark = pytest.mark.gpu


def far_rows(vocab, io):
    x, t = make(9, vocab, io, seed=7)
    x[0] = torch.finfo(x.dtype).min
    x[1] = -1e9
    x[2] = -1e4
    x[3] += 1e6                                      # differences that are left are exact
    x[4] = -math.inf
    x[4, 5:60] = torch.finfo(x.dtype).min
    x[5, :] = -3e4
    x[5, ::3] = -3e4 + 256
    x[6] *= 500
    x[7] = 1e30
    return x, t


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [61, 700, 40001])
def test_gradient(vocab, io, in_place):
    x, t = far_rows(vocab, io)
    rows, k = x.shape[0], 5
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    top = torch.randint(0, vocab, (rows, k), generator=gen, device="cuda", dtype=torch.int32)
    t[4], top[4] = 6, 7
    fwd = scores(x, t, 0, io)
    given = dict(d_logp=rnd(rows), d_entropy=rnd(rows), entropy=fwd["entropy"], top_tok=top, d_top_logp=rnd(rows, k))
    stride = x.shape[1] + 3 if in_place else None
    wide = torch.full((rows, vocab + 3), 50.0, dtype=x.dtype, device="cuda")
    wide[:, :vocab] = x
    into = wide[:, :vocab] if in_place else torch.full_like(x, 3.0)
    T.gdn_token_scores_backward(T.score_dims(rows, vocab, k, io, stride), into if in_place else x, t, fwd["lse"],
                                fwd["entropy"], given["d_logp"], given["d_entropy"], into, top, given["d_top_logp"])
    m = x.double().amax(1)
    shifted, lse = x.double() - m[:, None], fwd["lse"].double()
    check_gradient(shifted, t, into, given, io, torch.where(lse.abs() < 4096, lse - m, torch.logsumexp(shifted, 1)))
    assert (wide[:, vocab:] == 50).all()
