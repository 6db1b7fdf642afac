"""The gated delta rule in 64 bits, token by token, and its gradients by the chain rule of each token."""
import torch


def rel(x, ref):
    """2-norm of the difference over that of the reference; infinite where either is not finite."""
    x, ref = x.double().cpu().flatten(), ref.double().cpu().flatten()
    if not (torch.isfinite(x).all() and torch.isfinite(ref).all()):
        return float("inf")
    n = ref.norm().item()
    return (x - ref).norm().item() / n if n else (0.0 if not x.abs().max() else float("inf"))


def sequence(q, k, v, beta, g, S0, d_o=None, dS=None):
    """One sequence: q, k [n, hk, dk], v [n, hv, dv], beta, g [n, hv], S0 [hv, dv, dk].  Returns o and the end
    state and, with d_o, a dict of the gradients (dlog_g: of ln g)."""
    share = v.shape[1] // q.shape[1]
    q, k = (x.double().cpu().repeat_interleave(share, 1) for x in (q, k))
    v, beta, g, S = (x.double().cpu() for x in (v, beta, g, S0))
    n = v.shape[0]
    o, decayed = torch.zeros_like(v), []
    for t in range(n):
        P = g[t, :, None, None] * S
        w = v[t] - (P @ k[t, :, :, None])[..., 0]
        S = P + (beta[t, :, None] * w)[:, :, None] * k[t, :, None, :]
        o[t] = (S @ q[t, :, :, None])[..., 0]
        decayed.append((P, w, S))
    if d_o is None:
        return o, S
    d_o, dS = d_o.double().cpu(), torch.zeros_like(S) if dS is None else dS.double().cpu()
    out = {x: torch.zeros_like(y) for x, y in (("dq", q), ("dk", k), ("dv", v), ("dbeta", beta), ("dlog_g", g))}
    for t in reversed(range(n)):
        P, w, after = decayed[t]
        out["dq"][t] = (after.mT @ d_o[t, :, :, None])[..., 0]
        dS = dS + d_o[t, :, :, None] * q[t, :, None, :]
        along = (dS @ k[t, :, :, None])[..., 0]
        out["dbeta"][t] = (along * w).sum(-1)
        dw = beta[t, :, None] * along
        out["dv"][t] = dw
        out["dk"][t] = beta[t, :, None] * (dS.mT @ w[..., None])[..., 0] - (P.mT @ dw[..., None])[..., 0]
        dP = dS - dw[:, :, None] * k[t, :, None, :]
        out["dlog_g"][t] = (P * dP).sum((-1, -2))
        dS = g[t, :, None, None] * dP
    for x in ("dq", "dk"):
        out[x] = out[x].unflatten(1, (-1, share)).sum(2)
    out["dS0"] = dS
    return o, S, out


def batch(offsets, q, k, v, beta, g, S0=None, d_o=None, dS=None):
    """Packed sequences; results packed the same way (states stacked)."""
    off = [int(x) for x in offsets]
    shape = (v.shape[1], v.shape[2], q.shape[2])
    parts = []
    for b, (i, j) in enumerate(zip(off, off[1:])):
        s = torch.zeros(shape) if S0 is None else S0[b]
        parts.append(sequence(q[i:j], k[i:j], v[i:j], beta[i:j], g[i:j], s, None if d_o is None else d_o[i:j],
                              None if dS is None else dS[b]))
    got = dict(o=torch.cat([p[0] for p in parts]), S_out=torch.stack([p[1] for p in parts]))
    if d_o is not None:
        for x in ("dq", "dk", "dv", "dbeta", "dlog_g"):
            got[x] = torch.cat([p[2][x] for p in parts])
        got["dS0"] = torch.stack([p[2]["dS0"] for p in parts])
    return got
