"""What a sequence holds, or that it cannot be used, leaves the others' results as they are, to the bit."""
import pytest
import torch

from test_gpu_rule import ARGS, T, backward, forward, make, many

pytestmark = pytest.mark.gpu
ROWS = ("o", "dq", "dk", "dv", "dbeta", "dlog_g")


def batch(many_, io):
    return many(70, 2, 4, 128, 128, io=io) if many_ else make([40, 70, 20, 64], 1, 2, 64, 80, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("many_", [False, True])
def test_unusable_sequences_between_others(many_, io):
    """Two sequences more in the middle: one whose rows pass the tensor's, and one that goes back from there."""
    x = batch(many_, io)
    want, off, n = {**forward(x), **backward(x)}, x["offsets"].tolist(), x["q"].shape[0]
    at = 3
    y = {**x, "offsets": torch.tensor(off[:at] + [off[at - 1] if i else n + 500 for i in range(2)] + off[at:],
                                      dtype=torch.int32, device="cuda")}
    d = x["dims"]
    y["dims"] = T.rule_dims(d.batch + 2, d.h_k, d.h_v, d.d_k, d.d_v, io)
    put = lambda s: torch.cat([s[:at - 1], 0 * s[:2] + 5, s[at - 1:]])  # noqa: E731
    y.update(S0=put(x["S0"]), dS_out=put(x["dS_out"]))
    got = {**forward(y), **backward(y)}
    for name in ROWS:
        assert torch.equal(got[name], want[name]), name
    for name in ("S_out", "dS0"):
        assert torch.equal(got[name][:at - 1], want[name][:at - 1]) and torch.equal(got[name][at + 1:], want[name][at - 1:])
        assert (got[name][at - 1:at + 1] == 5).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("many_", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_elements_that_are_not_finite(many_, io, bad):
    x = batch(many_, io)
    want, b = {**forward(x), **backward(x)}, 2
    i, j = x["offsets"].tolist()[b:b + 2]
    assert j - i > 10
    for name in (*ARGS, "d_o"):
        y = {**x, name: x[name].clone()}
        y[name][j - 1] = bad
        got = {**forward(y), **backward(y)}
        for out in ROWS:
            assert torch.equal(got[out][:i], want[out][:i]) and torch.equal(got[out][j:], want[out][j:]), (name, out)
        for out in ("S_out", "dS0"):
            keep = [s for s in range(x["dims"].batch) if s != b]
            assert torch.equal(got[out][keep], want[out][keep]), (name, out)
