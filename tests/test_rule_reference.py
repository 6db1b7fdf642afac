"""The reference's gradients against differences of its own forward pass.  CPU only."""
import pytest
import torch

import rule_reference as R


@pytest.mark.parametrize("n,hk,hv,dk,dv", [(5, 1, 2, 4, 3), (7, 2, 2, 3, 5)])
def test_gradients_are_those_of_differences(n, hk, hv, dk, dv):
    g = torch.Generator().manual_seed(n)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x = dict(q=rnd(n, hk, dk), k=rnd(n, hk, dk), v=rnd(n, hv, dv), beta=torch.rand(n, hv, generator=g).double(),
             g=0.2 + 0.8 * torch.rand(n, hv, generator=g).double(), S0=rnd(hv, dv, dk))
    x["k"] /= x["k"].norm(dim=-1, keepdim=True)
    d_o, dS = rnd(n, hv, dv), rnd(hv, dv, dk)

    def value(**kw):
        o, S = R.sequence(**{**x, **kw})
        return ((o * d_o).sum() + (S * dS).sum()).item()
    got = R.sequence(**x, d_o=d_o, dS=dS)[2]
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("beta", "dbeta"), ("g", "dlog_g"), ("S0", "dS0")):
        along = rnd(*x[name].shape)
        if name == "g":
            step = lambda e: x["g"] * torch.exp(e * along)  # noqa: E731
        else:
            step = lambda e: x[name] + e * along  # noqa: E731
        h = 1e-5
        diff = (value(**{name: step(h)}) - value(**{name: step(-h)})) / (2 * h)
        want = (got[key] * along).sum().item()
        # central differences: h^2 of the third derivative, and 2^-53 of the value over h
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), name
