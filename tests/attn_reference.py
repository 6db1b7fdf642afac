"""Inputs and 64-bit references of the attention-layer tests (numpy, no GPU)."""
import numpy as np
import torch

EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}          # half a step, relative


def as_io(a, io):
    """float64 values of an array rounded to the element type, and the tensor itself (CPU)."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(torch.float32 if io == "f32" else torch.bfloat16)
    return t.to(torch.float64).numpy(), t


def parents(rng, kind, n):
    if kind == "chain":
        return np.arange(-1, n - 1)
    if kind == "star":
        return np.full(n, -1)
    return np.array([rng.integers(-1, i) if i else -1 for i in range(n)], dtype=np.int64)


def ancestors(par):
    """Strict ancestors, [n][n] booleans."""
    n = len(par)
    anc = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(par):
        if p >= 0:
            anc[i] = anc[p]
            anc[i, p] = True
    return anc


def pack_bits(anc, N):
    """[n][n] booleans -> int32 words [N][ceil(N / 32)], rows past n zero."""
    words = (N + 31) // 32
    full = np.zeros((N, words * 32), dtype=bool)
    full[:anc.shape[0], :anc.shape[1]] = anc
    return np.packbits(full, axis=-1, bitorder="little").view(np.uint32).view(np.int32)


def attend(q, keys, values, look, scale, io):
    """One sequence and key head in 64 bits.  q [n][group][d]; keys, values [L][d]; look [n][L].
    Returns o and an elementwise bound of the kernel's error, from its roundings: the fp32 sum of
    a score's d products and its exponential (delta, relative, on every weight), the fp32 sums over L
    keys, with bf16 elements the rounding of each weight (in numerator and denominator), and
    the rounding of the result."""
    d, L = keys.shape[-1], keys.shape[0]
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.einsum("ngd,ld->ngl", q, keys) * scale
        s = np.where(look[:, None, :], s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        w = p / p.sum(-1, keepdims=True)
        seen_v = np.where(np.isfinite(values), values, 0.0)
        o = np.einsum("ngl,ld->ngd", w, seen_v)
        mag = np.einsum("ngl,ld->ngd", w, np.abs(seen_v))
        qk = np.einsum("ngd,ld->ngl", np.abs(q), np.abs(np.where(look.any(0)[:, None], keys, 0.0)))
        qk = np.where(look[:, None, :], qk, 0.0).max(-1, keepdims=True) * scale
        delta = (d + 8) * 2.0 ** -24 * qk + 2.0 ** -21
        bound = (2 * delta + 2 * (L + 4) * 2.0 ** -24) * mag + EPS[io] * np.abs(o)
        if io == "bf16":
            bound += EPS[io] * (mag + np.abs(o)) * 1.01
        # values that are not finite reach the rows that see them
        for j in np.nonzero(~np.isfinite(values).all(-1))[0]:
            bad = np.where(np.isfinite(values[j]), 0.0, values[j])
            o = np.where(look[:, j][:, None, None], o + bad, o)
    return o, bound + 1e-30
