"""Rotary positions against their formula in 64 bits.  Error of an output: half a step of its type
relative to the value, and for the fp32 arithmetic before it half a step each of the cosine and sine
(times amp), the two products and their sum: at most 4 half steps of |x| + |y|."""
import numpy as np
import pytest
import torch

from attn_reference import EPS, as_io

pytestmark = pytest.mark.gpu
T = pytest.importorskip("tree_masked_gated_amd")


def turn(x, pos, freq, rot, layout, amp):
    """x [rows][heads][d] in 64 bits; the bound's |x| + |y| too."""
    angle = pos[:, None] * freq[None, :]
    c, s = np.cos(angle)[:, None, :] * amp, np.sin(angle)[:, None, :] * amp
    half = rot // 2
    a, b = (slice(0, half), slice(half, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    y, mag = x.copy(), np.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(amp)
    return y, mag


def case(sizes, N, hq, hkv, d, rot, layout, io, ctx, amp=1.0, ragged=False, freq=None, in_place=False, seed=0):
    print("[gpu-rope]", sizes, N, hq, hkv, d, rot, layout, io, amp, ragged, in_place, flush=True)
    rng = np.random.default_rng(seed)
    B, rows = len(sizes), sum(sizes)
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot) if freq is None else np.asarray(freq, np.float64)
    fused64, fused = as_io(rng.standard_normal((rows, hq + 2 * hkv, d)), io)
    depth = rng.integers(0, N, size=(B, N)).astype(np.int32)
    dev = "cuda"
    fused = fused.to(dev)
    off = np.concatenate([[0], np.cumsum(sizes)])
    pos = np.concatenate([ctx[b] + depth[b, :sizes[b]].astype(np.float64) for b in range(B)])
    q, k = fused[:, :hq], fused[:, hq:hq + hkv]
    qo, ko = (q, k) if in_place else (torch.empty((rows, hq, d), dtype=fused.dtype, device=dev),
                                      torch.empty((rows, hkv, d), dtype=fused.dtype, device=dev))
    T.gdn_attn_rope(T.attn_dims(B, N, hq, hkv, d, io), T.rope_dims(rot, layout, amp), q, k,
                    torch.from_numpy(freq).to(dev), torch.tensor(ctx, dtype=torch.int32, device=dev),
                    torch.from_numpy(depth).to(dev), qo, ko,
                    offsets=torch.from_numpy(off.astype(np.int32)).to(dev) if ragged else None)
    for x64, out in ((fused64[:, :hq], qo), (fused64[:, hq:hq + hkv], ko)):
        want, mag = turn(x64, pos, freq, rot, layout, amp)
        got = out.double().cpu().numpy()
        tol = EPS[io] * np.abs(want) * (io == "bf16") * 1.001 + 4 * EPS["f32"] * mag
        assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / (tol + 1e-300)).max())
    if in_place:
        assert np.array_equal(fused[:, hq + hkv:].double().cpu().numpy(), fused64[:, hq + hkv:])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(8, 2), (8, 8), (64, 32), (72, 20), (128, 128), (128, 64), (256, 64), (256, 250)])
def test_layouts(io, layout, d, rot):
    case([5, 5, 5], 5, 4, 2, d, rot, layout, io, [0, 17, 4000])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_far_positions_and_scaling(io):
    """Positions up to the largest, stretched frequencies, an amplitude."""
    case([3, 3], 3, 2, 1, 64, 64, "half", io, [1000000, 2 ** 31 - 8], amp=1.2079)
    case([3, 3], 3, 2, 1, 64, 64, "interleaved", io, [0, 131072], amp=0.5, freq=np.linspace(-3.0, 7.0, 32))


def test_ragged_and_in_place():
    case([0, 7, 1, 0, 64, 3], 64, 4, 2, 128, 64, "half", "bf16", [3, 0, 9, 2, 5000, 77], ragged=True)
    case([7, 1, 64], 64, 3, 1, 64, 64, "interleaved", "f32", [3, 0, 9], ragged=True, in_place=True)
    case([4, 4], 4, 4, 2, 64, 32, "half", "bf16", [3, 10], in_place=True)
    case([4, 4], 4, 4, 2, 64, 12, "half", "bf16", [3, 10], in_place=True)


def test_many_rows():
    """Four rows to a workgroup, the last one incomplete, and more sequences than a wave has lanes."""
    rng = np.random.default_rng(5)
    sizes = rng.integers(0, 40, size=150)
    sizes[0] = 40
    case(sizes.tolist(), 40, 8, 2, 64, 64, "half", "bf16", rng.integers(0, 9000, size=150).tolist(), ragged=True)
    case([41] * 51, 41, 2, 1, 128, 128, "interleaved", "bf16", rng.integers(0, 9000, size=51).tolist())


def test_invalid_tree_and_rows_of_nobody():
    d, dev = 64, "cuda"
    x = torch.randn(6, 3, d, device=dev)
    out_q, out_k = torch.full((6, 2, d), 7.0, device=dev), torch.full((6, 1, d), 7.0, device=dev)
    depth = torch.tensor([[-1, -1, -1], [0, 1, 2]], dtype=torch.int32, device=dev)
    T.gdn_attn_rope(T.attn_dims(2, 3, 2, 1, d, "f32"), T.rope_dims(32), x[:, :2], x[:, 2:],
                    torch.ones(16, dtype=torch.float64, device=dev), torch.tensor([5, 5], dtype=torch.int32, device=dev),
                    depth, out_q, out_k, offsets=torch.tensor([0, 2, 5], dtype=torch.int32, device=dev))
    for o in (out_q, out_k):
        assert torch.isnan(o[:2]).all() and torch.isfinite(o[2:5]).all() and (o[5] == 7.0).all()
