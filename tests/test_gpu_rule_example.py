"""The example's training and serving steps: the rule and the scores in their places among the tree's calls."""
import os
import sys

import pytest
import torch

import rule_reference as R

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def token_by_token(offsets, q, k, v, beta, log_g):
    """The rule as torch computes it on its own, for gradients."""
    share, out = v.shape[1] // q.shape[1], []
    q, k, g = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1), log_g.exp()
    for i, j in zip(offsets[:-1].tolist(), offsets[1:].tolist()):
        S = v.new_zeros(v.shape[1], v.shape[2], q.shape[2])
        for t in range(i, j):
            S = g[t, :, None, None] * S
            w = v[t] - (S @ k[t, :, :, None])[..., 0]
            S = S + (beta[t, :, None] * w)[:, :, None] * k[t, :, None, :]
            out.append((S @ q[t, :, :, None])[..., 0])
    return torch.stack(out)


def softmax_scores(logits, tokens):
    logp = torch.log_softmax(logits, -1)
    return logp.gather(1, tokens.long()[:, None])[:, 0], -(logp.exp() * logp).sum(-1)


def test_gradients_of_a_training_step():
    """Every parameter's gradient against torch's own in 64 bits.  A gradient passes the rule and its gradients (6e-6
    each), the scores' and the four products around them (sums of at most 208 terms, 15 roundings at random each:
    1e-6), 1.7e-5 together; normalisation and shared rows cancel no more than nine tenths of it: 1.7e-4."""
    from rule_train_and_serve import loss_of, train
    seen = []

    def check(s):
        p = {n: w.detach().double().cpu().requires_grad_(True) for n, w in s["p"].items()}
        want = loss_of(p, s["heads"], s["tokens"].cpu(), s["offsets"].cpu(), token_by_token, softmax_scores)
        want.backward()
        assert abs(s["loss"].item() - want.item()) <= 1e-5 * abs(want.item())
        for n, w in s["p"].items():
            assert R.rel(w.grad, p[n].grad) <= 1.7e-4, n
        seen.append(1)

    train(steps=2, on_step=check)
    assert len(seen) == 2


def test_serving_steps():
    """After every step the states are those of the prompt and all tokens so far, taken one by one, and so is the
    output of the last.  The tree's calls keep to 1e-2; the output is rounded to bf16."""
    from rule_train_and_serve import model, serve
    text, lengths = {}, []

    def check(s):
        off = s["offsets"].tolist()
        for b, (i, j) in enumerate(zip(off, off[1:])):
            path = s["path"][b, :int(s["path_len"][b])].tolist()
            assert int(s["accepted"][b]) == (path[-1] if path else -1) and int(s["accept_len"][b]) == len(path)
            assert all(int(s["drafted"][b, n]) == int(s["root"][b] if a is None else s["target"][b, a])
                       for a, n in zip([None] + path, path))
            text.setdefault(b, s["prompt"][i:j].tolist())
            text[b] += s["drafted"][b, path].tolist() + [int(s["token"][b])]
            q, k, v, beta, g = s["rows"](torch.tensor(text[b], device="cuda"))
            o, S = R.sequence(q, k, v, beta, g, torch.zeros_like(s["state"][b]))
            assert R.rel(s["state"][b], S) <= 1e-2 and R.rel(s["last"][b], o[-1]) <= 1e-2 + 2.0 ** -8
        lengths.append(s["path_len"].tolist())

    serve(*model(), steps=3, on_step=check)
    assert len(lengths) == 3 and max(map(max, lengths)) > 0
