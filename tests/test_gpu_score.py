"""Scores of tokens on the GPU, against 64 bits.

Tolerances.  A log-probability is (x - m) - ln s: x - m is rounded to 2^-24 of itself, s is a sum of up
to 2^17 terms of random rounding (2^-24 each, less than 2^-24 sqrt(17) through the tree of sums, and
2^-22 for the exponential), so ln s is within 2^-21, absolutely, and lse within that and 2^-24 of
itself.  The entropy's mean adds 2^-22 of values up to ln(vocab) < 13: 4e-6.  A gradient's p is the
exponential of l = x - lse, which is rounded to 2^-24 |l|, and so is its multiple by log2 e; with the
exponential's own 2^-23 that is (2 |l| + 2) 2^-24 of p, and l enters the entropy's part once more,
with 2^-24 |l|.  (32 + 4 |l|) 2^-24 of the parts' sizes covers these and the sums; bf16 adds half a
step, 2^-8.
"""
import math

import pytest
import torch

T = pytest.importorskip("tree_masked_gated_amd")
pytestmark = pytest.mark.gpu

LOG, ENT = 2.0 ** -21, 4e-6


def scores(x, tokens, k, io, stride=None, ws=None, stream=None):
    n, v = x.shape
    d = T.score_dims(n, v, k, io, stride)
    f = lambda *s: torch.full(s, 77.0, device="cuda")  # noqa: E731
    out = dict(logp=f(n), entropy=f(n), lse=f(n))
    top = dict(top_logp=f(n, k), top_tok=torch.full((n, k), -9, dtype=torch.int32, device="cuda")) if k else {}
    ws = T.score_workspace(d) if ws is None else ws
    T.gdn_token_scores(d, x, tokens, out["logp"] if tokens is not None else None, out["entropy"], out["lse"], ws, **top,
                       stream=stream)
    return {**out, **top}


def reference(x, tokens, k):
    x = x.double()
    logp = torch.log_softmax(x, 1)
    p = logp.exp()
    out = dict(entropy=-torch.xlogy(p, p).sum(1), lse=torch.logsumexp(x, 1))
    if tokens is not None:
        out["logp"] = logp.gather(1, tokens.long()[:, None])[:, 0]
    order = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices[:, :k]
    return {**out, "top_tok": order.int(), "top_logp": logp.gather(1, order)}


def close(got, want, absolute, relative=2.0 ** -23):
    got, want = got.double(), want.double()
    finite = torch.isfinite(want)
    assert torch.equal(finite, torch.isfinite(got)) and torch.equal(got[~finite], want[~finite])
    assert ((got - want)[finite].abs() <= absolute + relative * want[finite].abs()).all()


def check(x, tokens, k, got):
    want = reference(x, tokens, k)
    close(got["lse"], want["lse"], LOG)
    close(got["entropy"], want["entropy"], ENT)
    if tokens is not None:
        close(got["logp"], want["logp"], LOG)
    if k:
        assert torch.equal(got["top_tok"], want["top_tok"])
        close(got["top_logp"], want["top_logp"], LOG)


def make(rows, vocab, io, seed=0, std=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * std).to(torch.float32 if io == "f32" else torch.bfloat16)
    return x, torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (3, 2, 2), (5, 7, 0), (2, 64, 64), (4, 100, 8), (7, 513, 1),
                                          (600, 1000, 3), (2, 32000, 8), (1, 131073, 64), (33, 10007, 5),
                                          (3, 50001, 20), (1, 8193, 1), (520, 4099, 64)])
def test_scores(rows, vocab, k, io):
    x, t = make(rows, vocab, io)
    check(x, t, k, scores(x, t, k, io))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(3, 40000), (700, 900)])
def test_masks_and_ties(rows, vocab, io):
    """Most or all but a few entries masked, by -inf or by the type's lowest value; rows of equal logits; zeros of
    both signs: more elements than fit reach any bound."""
    x, t = make(rows, vocab, io)
    low = torch.finfo(x.dtype).min
    x[0] = 1.5
    x[1, 5:] = -math.inf
    x[1, 700] = 2.0
    x[2, :] = low
    x[2, 3::200] = 1.0
    t[1] = 700
    for k in (0, 1, 4, 64):
        check(x, t, k, scores(x, t, k, io))
    x[0] = low
    x[1] = 0.0
    x[1, ::3] = -0.0
    x[2] = torch.arange(vocab, device="cuda").to(x.dtype) / 50 - 30     # ascending: many equal in bf16
    for k in (1, 64):
        check(x, t, k, scores(x, t, k, io))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_without_a_distribution(io):
    """No finite logit, +inf, NaN: results as the formulas give them, other rows untouched, and alternatives in
    order all the same, NaN first."""
    x, t = make(5, 20000, io)
    x[1] = -math.inf
    x[2, 77] = math.inf
    x[3, 5000] = math.nan
    x[3, 9] = math.nan
    got = scores(x, t, 3, io)
    keep = [0, 4]
    check(x[keep], t[keep], 3, {a: b[keep] for a, b in got.items()})
    assert all(got[a][1:4].isnan().all() for a in ("entropy", "logp"))
    assert got["lse"][[1, 3]].isnan().all() and not torch.isfinite(got["lse"][2])
    assert got["top_tok"][1].tolist() == [0, 1, 2] and got["top_tok"][2, 0] == 77
    assert got["top_tok"][3, :2].tolist() == [9, 5000]
    best = x[3].float().nan_to_num(-100).argmax()
    assert got["top_tok"][3, 2] == best


def test_what_is_not_wanted_and_tokens_outside():
    x, t = make(4, 300, "f32")
    d = T.score_dims(4, 300, 0, "f32")
    lse = torch.empty(4, device="cuda")
    T.gdn_token_scores(d, x, None, None, None, lse, T.score_workspace(d))
    close(lse, torch.logsumexp(x.double(), 1), LOG)
    t[1], t[2] = -1, 300
    got = scores(x, t, 0, "f32")
    assert got["logp"][1:3].isnan().all() and torch.isfinite(got["logp"][[0, 3]]).all()
    T.gdn_token_scores(T.score_dims(0, 300, 0, "f32"), x[:0], None, None, None, lse[:0], T.score_workspace(d))


@pytest.mark.parametrize("io,stride,skip", [("bf16", 1000, 0), ("f32", 777, 0), ("bf16", 1001, 8), ("f32", 700, 4)])
def test_strides(io, stride, skip):
    """Rows at any distance, and what lies between them: neither read into a result nor written."""
    x, t = make(6, 690, io)
    wide = torch.full((6 * stride + 16,), 50.0, dtype=x.dtype, device="cuda")
    view = wide[skip:skip + 6 * stride].view(6, stride)[:, :690]
    view.copy_(x)
    check(x, t, 4, scores(view, t, 4, io, stride))
    d = T.score_dims(6, 690, 0, io, stride)
    lse, g = torch.logsumexp(x.float(), 1), torch.ones(6, device="cuda")
    before = wide.clone()
    T.gdn_token_scores_backward(d, view, t, lse, None, g, None, view)          # in the logits' place
    between = torch.ones_like(wide, dtype=torch.bool)
    between[skip:skip + 6 * stride].view(6, stride)[:, :690] = False
    assert torch.equal(wide[between], before[between])
    check_gradient(x, t, view, dict(d_logp=g), io, lse)


def check_gradient(x, t, got, given, io, lse):
    x = x.double()
    far = (x - lse.double()[:, None]).abs().clamp(max=200)           # p is 0 beyond
    p = torch.exp(x - lse.double()[:, None])
    d, extra = torch.zeros_like(x), torch.zeros_like(x)
    if "d_entropy" in given:
        h = given["entropy"].double()[:, None]
        extra = torch.where(p > 0, -p * given["d_entropy"].double()[:, None] * (torch.where(p > 0, p, 1).log() + h), 0.0)
    if "d_logp" in given:
        ok = (t >= 0) & (t < x.shape[1])
        d[ok] = d[ok].scatter_add(1, t[ok].long()[:, None], given["d_logp"][ok].double()[:, None])
    if "top_tok" in given:
        for r in range(x.shape[0]):
            for tok, val in zip(given["top_tok"][r].tolist(), given["d_top_logp"][r].tolist()):
                if 0 <= tok < x.shape[1]:
                    d[r, tok] += val
    want = d - p * d.sum(1, keepdim=True) + extra
    # the parts are rounded each by itself, and cancel only in their sum
    size = d.abs() + p * d.abs().sum(1, keepdim=True) + extra.abs()
    if "d_entropy" in given:
        size = size + p * given["d_entropy"].double().abs()[:, None] * (1 + given["entropy"].double()[:, None])
    step = 0.0 if io == "f32" else 2.0 ** -8
    # values below the smallest normal one (2^-126) may be flushed
    assert ((got.double() - want).abs() <= step * want.abs() + (32 + 4 * far) * 2.0 ** -24 * size + 2.0 ** -126).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (3, 100, 0), (40, 5001, 8), (2, 70000, 64), (5, 16385, 4)])
def test_gradient(rows, vocab, k, io):
    x, t = make(rows, vocab, io)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    if vocab > 50:
        x[:, vocab - 3:] = -math.inf
        x[0, 10:20] = torch.finfo(x.dtype).min
    fwd = scores(x, t, 0, io)
    given = dict(d_logp=rnd(rows), d_entropy=rnd(rows), entropy=fwd["entropy"])
    if k:
        top = torch.randint(0, vocab, (rows, k), generator=gen, device="cuda", dtype=torch.int32)
        top[:, 0] = t                                # the token among its alternatives
        if k > 3:
            top[:, 1] = top[:, 2]                    # a token twice
            top[0, 3], top[-1, 3] = -1, vocab        # and none
        given.update(top_tok=top, d_top_logp=rnd(rows, k))
    d, out = T.score_dims(rows, vocab, k, io), torch.full_like(x, 3.0)
    T.gdn_token_scores_backward(d, x, t, fwd["lse"], fwd["entropy"], given["d_logp"], given["d_entropy"], out,
                                given.get("top_tok"), given.get("d_top_logp"))
    check_gradient(x, t, out, given, io, fwd["lse"])
    T.gdn_token_scores_backward(d, x, None, fwd["lse"], fwd["entropy"], None, given["d_entropy"], out)
    check_gradient(x, t, out, dict(d_entropy=given["d_entropy"], entropy=fwd["entropy"]), io, fwd["lse"])


def test_gradient_is_that_of_differences():
    """The calls against each other, fp32: along a random direction of unit length the scores move by the
    gradient's product with it; a step of 1/16 leaves (1/16)^2 / 6 of a third derivative below 4, and the
    scores' rounding, 3e-6, over the step."""
    x, t = make(6, 500, "f32", std=1.0)
    gen = torch.Generator(device="cuda").manual_seed(2)
    gl, ge = (torch.randn(6, generator=gen, device="cuda") for _ in range(2))
    f, out = scores(x, t, 0, "f32"), torch.empty_like(x)
    T.gdn_token_scores_backward(T.score_dims(6, 500, 0, "f32"), x, t, f["lse"], f["entropy"], gl, ge, out)
    for _ in range(4):
        along = torch.randn(x.shape, generator=gen, device="cuda")
        along /= along.norm(dim=1, keepdim=True)
        a, b = (scores(x + e * along, t, 0, "f32") for e in (1 / 16, -1 / 16))
        diff = sum((g * (a[n] - b[n]) * 8 for g, n in ((gl, "logp"), (ge, "entropy"))))
        want = (out * along).sum(1)
        assert ((diff - want).abs() <= (4 / 6 / 256 + 16 * 3e-6) * (gl.abs() + ge.abs())).all()


def test_runs_alike_streams_graphs_and_shared_workspace():
    """The same bits from run to run, on a stream of its own, with a workspace full of other numbers, and from a
    captured graph replayed among other calls."""
    x, t = make(3, 60001, "bf16")
    first = scores(x, t, 16, "bf16")
    d = T.score_dims(3, 60001, 16, "bf16")
    ws = torch.full((T.gdn_score_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = scores(x, t, 16, "bf16", ws=ws)
    side.synchronize()
    for name in first:
        assert torch.equal(first[name], again[name]), name
    out = {a: torch.empty_like(b) for a, b in first.items()}
    grad, g = torch.empty_like(x), torch.ones(3, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.gdn_token_scores(d, x, t, out["logp"], out["entropy"], out["lse"], ws, out["top_logp"], out["top_tok"])
        T.gdn_token_scores_backward(d, x, t, out["lse"], out["entropy"], g, g, grad, out["top_tok"], out["top_logp"])
    kept = None
    for _ in range(3):
        for v in (*out.values(), grad):
            v.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for name in first:
            assert torch.equal(first[name], out[name]), name
        assert kept is None or torch.equal(kept, grad)
        kept = grad.clone()
        scores(*make(2, 40000, "bf16", seed=9), 16, "bf16", ws=ws)


def test_rows_past_two_to_the_32_bytes():
    """A row that begins past 2^32 bytes."""
    n = 2 ** 31 // 65536 + 2
    x = torch.zeros(n, 65536, dtype=torch.bfloat16, device="cuda")
    x[-1], x[0] = make(1, 65536, "bf16")[0][0], 1.0
    t = torch.full((n,), 9, dtype=torch.int32, device="cuda")
    got = scores(x, t, 2, "bf16")
    check(x[-1:], t[-1:], 2, {a: b[-1:] for a, b in got.items()})
    g = torch.ones(n, device="cuda")
    T.gdn_token_scores_backward(T.score_dims(n, 65536, 0, "bf16"), x, t, got["lse"], None, g, None, x)
    check_gradient(make(1, 65536, "bf16")[0], t[-1:], x[-1:], dict(d_logp=g[-1:]), "bf16", got["lse"][-1:])
