"""Up to 16 rows of a key head with bf16 elements: the weights keep 2^-16, so that what is left is the fp32
arithmetic and the rounding of the result."""
import numpy as np
import pytest

from attn_reference import EPS, attend
from test_gpu_attn_verify import Case

pytestmark = pytest.mark.gpu


def check(c, o):
    """Bound: as attend() for fp32 elements, and the roundings to bf16: half a step of the result, and of each weight
    (in numerator and denominator) that of the rest which its first term leaves, 2^-8 of 2^-8 of it."""
    got = o.double().cpu().numpy()
    for b in range(c.B):
        n, x = c.sizes[b], c.fused64[c.starts[b]:c.starts[b] + c.sizes[b]]
        look = np.concatenate([np.ones((n, c.ctx[b]), dtype=bool), c.anc[b] | np.eye(n, dtype=bool)], axis=1)
        for h in range(c.hkv):
            q = x[:, h * c.group:(h + 1) * c.group]
            keys = np.concatenate([c.prefix[b][0][:, h], x[:, c.hq + h]])
            values = np.concatenate([c.prefix[b][1][:, h], x[:, c.hq + c.hkv + h]])
            want, tol = attend(q, keys, values, look, c.scale, "f32")
            mag, _ = attend(q, keys, np.abs(values), look, c.scale, "f32")
            tol = tol + EPS["bf16"] * np.abs(want) * 1.001 + EPS["bf16"] ** 2 * (mag + np.abs(want)) * 1.01
            err = np.abs(got[c.starts[b]:c.starts[b] + n, h * c.group:(h + 1) * c.group] - want)
            assert (err <= tol).all(), (b, h, float((err / tol).max()))


@pytest.mark.parametrize("d", [8, 64, 72, 128, 256])
@pytest.mark.parametrize("qstd", [0.5, 2.0])
def test_tokens(d, qstd):
    print("[gpu-attn-tokens]", d, qstd, flush=True)
    c = Case([1] * 6, [0, 1, 31, 130, 700, 3000], "star", 8, 2, d, "bf16", 16, qstd=qstd)
    check(c, c.call())


@pytest.mark.parametrize("n,hq,hkv,kind", [(16, 2, 2, "chain"), (4, 8, 2, "rrt"), (5, 3, 1, "rrt"), (2, 8, 1, "star")])
def test_small_trees(n, hq, hkv, kind):
    print("[gpu-attn-tokens]", n, hq, hkv, kind, flush=True)
    c = Case([n] * 4, [0, 45, 1000, 130], kind, hq, hkv, 128, "bf16", 24)
    check(c, c.call())


def test_one_long_context():
    c = Case([1], [40000], "star", 8, 1, 128, "bf16", 16)
    check(c, c.call())
