"""The rule where offsets pass 32 bits: rows far apart, pools and workspaces of more than 2^32 bytes."""
import pytest
import torch

from test_gpu_rule import ARGS, F32, R, T, backward, bound, check, forward, grads_like, make

pytestmark = pytest.mark.gpu
ROWS = ("q", "k", "v", "d_o")


def far(x, stride):
    """The same values in memory of their own, rows `stride` elements apart."""
    n, heads, width = x.shape
    y = torch.empty((n - 1) * stride + heads * width, dtype=x.dtype, device="cuda").as_strided(x.shape, (stride, width, 1))
    return y.copy_(x)


@pytest.mark.parametrize("io,batch", [("bf16", 2), ("f32", 2), ("bf16", 70)])
def test_rows_past_two_to_the_32_bytes(io, batch):
    """The results of the same rows close together."""
    sizes = [66, 5] + [0] * (batch - 2)
    x = make(sizes, 2, 4, 128, 128, io)
    want = {**forward(x), **backward(x)}
    stride = 2 ** 25 + 8 if io == "bf16" else 2 ** 24 + 8
    assert 70 * stride * x["q"].element_size() > 2 ** 32
    y = {**x, **{a: far(x[a], stride) for a in ROWS}}
    f = forward(y, o=far(torch.zeros_like(x["v"]), stride))
    grads = {a: far(g, stride) if a in ("dq", "dk", "dv") else g for a, g in grads_like(x).items()}
    for name, value in {**f, **backward(y, out=grads)}.items():
        assert torch.equal(value, want[name]), name


def test_step_rows_and_pool():
    """Tokens whose rows lie far apart, states of a pool of more than 2^32 bytes."""
    x = make([1] * 70, 2, 4, 128, 128, "bf16")
    n = 2 ** 32 // (4 * 128 * 128 * 4) + 70
    pool, slot = torch.empty(n, 4, 128, 128, device="cuda"), torch.arange(n - 70, n, dtype=torch.int32, device="cuda")
    pool[n - 70:] = x["S0"]
    want, S, o = torch.empty_like(x["v"]), x["S0"].clone(), far(torch.zeros_like(x["v"]), 2 ** 25 + 8)
    T.gdn_rule_step(x["dims"], *(x[a] for a in ARGS), S, want)
    y = {**x, **{a: far(x[a], 2 ** 25 + 8) for a in ("q", "k", "v")}}
    T.gdn_rule_step(x["dims"], *(y[a] for a in ARGS), pool, o, slot=slot)
    assert torch.equal(o, want) and torch.equal(pool[n - 70:], S)


def test_a_long_batch():
    """A short sequence behind one of 2^17 rows, whose workspace passes 2^32 bytes: the results that it has by
    itself, and those of the 64-bit rule."""
    n, last = 2 ** 17, 70
    x = make([n, last], 32, 32, 128, 128, "bf16")
    assert T.gdn_rule_workspace_bytes(x["dims"], n + last) > 2 ** 32
    got = {**forward(x), **backward(x)}
    alone = {a: x[a][n:].contiguous() for a in (*ARGS, "d_o")}
    alone.update(S0=x["S0"][1:].contiguous(), dS_out=x["dS_out"][1:].contiguous(), dims=T.rule_dims(1, 32, 32, 128, 128, "bf16"),
                 offsets=torch.tensor([0, last], dtype=torch.int32, device="cuda"))
    tail = {a: v[1:] if a in ("S_out", "dS0") else v[n:] for a, v in got.items()}
    check(alone, tail, "bf16")
    for name, value in {**forward(alone), **backward(alone)}.items():
        assert R.rel(tail[name], value) <= 2 * bound(name, "bf16") + F32, name
    for name, value in got.items():
        assert torch.isfinite(value).all(), name
