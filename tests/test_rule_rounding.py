"""The bounds of rule_rounding on the CPU: they hold for two terms of every factor that has two, and no factor's single
term keeps to them."""
import pytest
import torch

import rule_reference as R
import rule_rounding as Q


@pytest.fixture(scope="module")
def case():
    gen = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    n, hk, hv, d = 217, 1, 2, 64
    x = dict(q=rnd(n, hk, d) * d ** -0.5, k=torch.nn.functional.normalize(rnd(n, hk, d), dim=-1), v=rnd(n, hv, d),
             d_o=rnd(n, hv, d))
    x = {a: b.bfloat16() for a, b in x.items()}
    x.update(beta=torch.rand(n, hv, generator=gen), g=torch.exp(-torch.logspace(-3, 0, hv) * torch.rand(n, hv, generator=gen)),
             S0=0.3 * rnd(2, hv, d, d), dS_out=0.3 * rnd(2, hv, d, d), offsets=torch.tensor([0, 200, n]))
    want = R.batch(x["offsets"].tolist(), *(x[a] for a in ("q", "k", "v", "beta", "g")), x["S0"], x["d_o"], x["dS_out"])
    return x, want, Q.parts(x)


FACTORS = {"o": ("H", "U", "Y"), "dk": ("P", "G", "dkU", "dH")}


def rounded(p, name):
    return p[name].sum(0).bfloat16()


@pytest.mark.parametrize("name", FACTORS)
def test_parts_are_the_rule(case, name):
    assert R.rel(case[2][name].sum(0), case[1][name]) <= 1e-12


@pytest.mark.parametrize("name", FACTORS)
def test_two_terms_keep_to_the_bound(case, name):
    x, want, p = case
    got = Q.parts(x, {f: 2 for f in FACTORS[name]})
    assert Q.from_rounded(rounded(got, name), want[name]) <= Q.bound(name, p)


@pytest.mark.parametrize("name,factor", [(n, f) for n in FACTORS for f in FACTORS[n]])
def test_one_term_does_not(case, name, factor):
    x, want, p = case
    got = Q.parts(x, {f: 1 if f == factor else 2 for f in FACTORS[name]})
    assert Q.from_rounded(rounded(got, name), want[name]) > 1.3 * Q.bound(name, p)
