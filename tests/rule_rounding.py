"""Where bf16 rows of the rule are rounded: the chunked form in 64 bits, with chosen factors as sums of bf16 terms.

Products that reach bf16 rows alone take two terms of their fp32 factors: H, U and Y in o, P^T, G, U and dH' in dk.
Two terms leave 2^-16 of a factor; a product of two such factors has two of these, and the product of the
second terms, 2^-16 again, is left out: at most 3 2^-16 of a part of the result, the parts' errors at random to
each other.  With fp32's part of F32 a result is within `before` of 64 bits before its one rounding:

    before = 3 2^-16 |parts|_2 / |result|_2 + F32

Then it is rounded once.  Two numbers that are d apart round to different ones in d / step of the cases, and
then are a step apart, at most 2^-7 of the value: in the 2-norm sqrt(2^-7 before) of the result, beside `before`
itself.  So it lies within `bound` of the 64-bit result rounded once, where a factor of one term would leave
several times that."""
import torch

import rule_reference as R

C, F32 = 64, 6e-6


def split(x, terms):
    """x as the sum of this many bf16 terms (None: x itself)."""
    if terms is None:
        return x
    out = torch.zeros_like(x)
    for _ in range(terms):
        out = out + (x - out).bfloat16().double()
    return out


def head(q, k, v, beta, g, S0, d_o, dS, terms):
    """One value head of one sequence: the parts of o and those of dk."""
    n, H, kept, o = v.shape[0], S0.T.clone(), [], []
    t = lambda name, x: split(x, terms.get(name))  # noqa: E731
    for i in range(0, n, C):
        s = slice(i, min(i + C, n))
        G = g[s].log().cumsum(0)
        a, e, D = G.exp()[:, None], (G[-1] - G).exp()[:, None], (G[:, None] - G).tril().exp().tril()
        L, Y = (D * (k[s] @ k[s].T)).tril(-1), D * (q[s] @ k[s].T)
        W = torch.linalg.solve_triangular(torch.eye(len(G)).double() + L * beta[s], v[s] - a * (k[s] @ H), upper=False)
        U = beta[s, None] * W
        o.append(torch.stack([a * (q[s] @ t("H", H)), t("Y", Y) @ t("U", U)]))
        kept.append((s, H, U, a, e, D, L, Y))
        H = a[-1] * H + k[s].T @ (e * U)
    dH, dk = dS.T.clone(), []
    for s, H, U, a, e, D, L, Y in reversed(kept):
        b = beta[s, None]
        dU = Y.T @ d_o[s] + e * (k[s] @ dH)
        dR = torch.linalg.solve_triangular((torch.eye(len(b)).double() + b * L).T, dU, upper=True)
        P, G = D * (d_o[s] @ U.T), -(b * D * (dR @ U.T)).tril(-1)
        P, G = t("P", P.T), t("G", G + G.T)
        dk.append(torch.stack([P @ q[s], G @ k[s], e * (t("dkU", U) @ t("dH", dH).T), -a * b * (dR @ H.T)]))
        dH = a[-1] * dH + q[s].T @ (a * d_o[s]) - k[s].T @ (a * b * dR)
    return torch.cat(o, 1), torch.cat(dk[::-1], 1)


def parts(x, terms={}):
    """o's parts [2, rows, h_v, d_v] and dk's [4 h_v / h_k, rows, h_k, d_k] of packed sequences."""
    y = {a: x[a].double().cpu() for a in ("q", "k", "v", "beta", "g", "S0", "d_o", "dS_out")}
    off, share = x["offsets"].tolist(), x["v"].shape[1] // x["q"].shape[1]
    o, dk = [], []
    for b, (i, j) in enumerate(zip(off, off[1:])):
        if i == j:
            continue
        heads = [head(y["q"][i:j, h // share], y["k"][i:j, h // share], y["v"][i:j, h], y["beta"][i:j, h], y["g"][i:j, h],
                      y["S0"][b, h], y["d_o"][i:j, h], y["dS_out"][b, h], terms) for h in range(y["v"].shape[1])]
        o.append(torch.stack([p[0] for p in heads], 2))
        dk.append(torch.stack([torch.cat([heads[h + s][1] for s in range(share)]) for h in range(0, len(heads), share)], 2))
    return dict(o=torch.cat(o, 1), dk=torch.cat(dk, 1))


def bound(name, p):
    """p: the parts of o and dk.  dq's and dv's factors have three terms."""
    before = F32
    if name in p:
        before += 3 * 2.0 ** -16 * (p[name].norm() / p[name].sum(0).norm()).item()
    return (2.0 ** -7 * before) ** 0.5 + before


def from_rounded(got, want):
    return R.rel(got, want.to(torch.bfloat16))
