"""Tree attention over a paged cache against a 64-bit reference, element by element within the
bound that its roundings give (attn_reference.attend)."""
import numpy as np
import pytest
import torch

from attn_reference import ancestors, as_io, attend, pack_bits, parents

pytestmark = pytest.mark.gpu
T = pytest.importorskip("tree_masked_gated_amd")


class Case:
    """A batch of trees over a paged cache, on the host (64 bits) and on the device."""

    def __init__(self, sizes, ctx, kind, hq, hkv, d, io, page, order="rows", ragged=False, seed=0, N=None,
                 slack=1, garbage=float("nan"), qstd=2.0):
        rng = np.random.default_rng(seed)
        self.sizes, self.ctx, self.io = list(sizes), list(ctx), io
        self.hq, self.hkv, self.d, self.group = hq, hkv, d, hq // hkv
        B = self.B = len(ctx)
        N = self.N = N or max(max(sizes), 1)
        self.offsets = np.concatenate([[0], np.cumsum(sizes)])
        rows = int(self.offsets[-1])
        self.starts = self.offsets[:-1]
        dev = "cuda"
        self.par = [parents(rng, kind, n) for n in sizes]
        self.anc = [ancestors(p) for p in self.par]
        self.anc_dev = torch.from_numpy(np.stack([pack_bits(a, N) for a in self.anc])).to(dev)
        self.status = torch.zeros(B, dtype=torch.int32, device=dev)
        # one projection's output: q, k and v are slices of it
        fused = rng.standard_normal((rows, hq + 2 * hkv, d))
        fused[:, :hq] *= qstd
        self.fused64, t = as_io(fused, io)
        self.fused = t.to(dev)
        held = [-(-c // page) for c in ctx]
        width = max(max(held), 1) + slack
        n_pages = sum(held) + 3
        ids = rng.permutation(n_pages)
        self.table = np.full((B, width), -1, dtype=np.int32)
        pool = np.full((2, n_pages, page, hkv, d), garbage)
        self.prefix = []
        at = 0
        for b, c in enumerate(ctx):
            mine = ids[at:at + held[b]]
            at += held[b]
            self.table[b, :held[b]] = mine
            kv64, _ = as_io(rng.standard_normal((2, c, hkv, d)), io)
            self.prefix.append(kv64)
            for j in range(c):
                pool[:, mine[j // page], j % page] = kv64[:, j]
        self.pools = []
        for x in pool:
            _, t = as_io(x, io)
            if order == "heads":
                t = t.transpose(1, 2).contiguous().to(dev).transpose(1, 2)
            else:
                t = t.to(dev)
            self.pools.append(t)
        self.ctx_dev = torch.tensor(ctx, dtype=torch.int32, device=dev)
        self.table_dev = torch.from_numpy(self.table).to(dev)
        self.off_dev = torch.from_numpy(self.offsets.astype(np.int32)).to(dev) if ragged else None
        self.scale = d ** -0.5
        self.rows = rows
        self.dims = T.attn_dims(B, N, hq, hkv, d, io, self.scale)
        self.cache = T.PagedCache(*self.pools)
        self.ws = T.attn_workspace(self.dims)

    def call(self, o=None):
        o = torch.full((self.rows, self.hq, self.d), 7.0, dtype=self.fused.dtype, device="cuda") if o is None else o
        hq, hkv = self.hq, self.hkv
        T.gdn_attn_verify(self.dims, self.cache, self.table_dev, self.ctx_dev, self.fused[:, :hq],
                          self.fused[:, hq:hq + hkv], self.fused[:, hq + hkv:], self.anc_dev, self.status, o,
                          self.ws, offsets=self.off_dev)
        return o

    def check(self, o, skip=()):
        got = o.double().cpu().numpy()
        assert int(self.ws[:self.B * 4].view(torch.int32).abs().sum()) == 0      # counters are back at zero
        for b in range(self.B):
            n, c = self.sizes[b], self.ctx[b]
            if n == 0 or b in skip:
                continue
            r = slice(self.starts[b], self.starts[b] + n)
            x = self.fused64[r]
            look = np.concatenate([np.ones((n, c), dtype=bool), self.anc[b] | np.eye(n, dtype=bool)], axis=1)
            for h in range(self.hkv):
                q = x[:, h * self.group:(h + 1) * self.group]
                keys = np.concatenate([self.prefix[b][0][:, h], x[:, self.hq + h]])
                values = np.concatenate([self.prefix[b][1][:, h], x[:, self.hq + self.hkv + h]])
                want, tol = attend(q, keys, values, look, self.scale, self.io)
                have = got[r, h * self.group:(h + 1) * self.group]
                fine = np.isfinite(want)
                assert np.array_equal(fine, np.isfinite(have)), (b, h)
                assert np.array_equal(np.isnan(want), np.isnan(have)), (b, h)
                err = np.abs(np.where(fine, have - np.where(fine, want, 0), 0))
                assert (err <= tol).all(), (b, h, float((err / tol).max()))


def run(*args, **kw):
    print("[gpu-attn]", args, kw, flush=True)
    c = Case(*args, **kw)
    o = c.call()
    torch.cuda.synchronize()
    c.check(o)
    again = c.call()
    assert torch.equal(o.view(torch.uint8), again.view(torch.uint8))     # the same bits, whoever arrives last
    return c, o


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 64, 72, 128, 136, 256])
def test_token(io, d):
    """The next token alone: contexts from nothing to several shares."""
    run([1] * 6, [0, 1, 31, 32, 130, 700], "star", 4, 2, d, io, 16)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (8, 1), (6, 2), (48, 3)])
def test_heads(io, hq, hkv):
    run([1, 5, 3], [45, 0, 200], "rrt", hq, hkv, 64, io, 24, ragged=True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [2, 8, 13, 16, 17, 32, 33, 64, 65, 130])
def test_tree_sizes(io, n):
    """Every shape of the row tiles, both tree extremes and a random one."""
    kind = {0: "rrt", 1: "chain", 2: "star"}[n % 3]
    run([n, n], [70, 3], kind, 4, 2, 128, io, 16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,hq", [(16, 2), (20, 2), (40, 2), (33, 8), (90, 8)])
def test_rows_and_widths(d, n, hq):
    run([n, n - 1, 1], [300, 64, 129], "rrt", hq, 2, d, "bf16", 32, ragged=True)


@pytest.mark.parametrize("page", [1, 5, 16, 24, 128, 1000])
@pytest.mark.parametrize("order", ["rows", "heads"])
def test_pages(page, order):
    run([9, 9], [257, 40], "rrt", 4, 2, 64, "bf16", page, order=order)


def test_large_tree():
    run([1024], [100], "rrt", 2, 1, 64, "bf16", 16)


def test_ragged_with_empty_sequences():
    run([0, 7, 0, 77, 1, 0], [5, 0, 0, 500, 2001, 9], "rrt", 8, 4, 64, "f32", 24, ragged=True, N=80)
    run([0, 7, 0, 77, 1, 0], [5, 0, 0, 500, 2001, 9], "rrt", 8, 4, 64, "bf16", 24, ragged=True, N=80)


def test_one_long_context():
    """One sequence whose keys are cut into the most parts."""
    run([1], [40000], "star", 8, 1, 64, "bf16", 16)
    run([3], [20011], "star", 2, 2, 128, "f32", 16)


def test_many_sequences():
    """More sequences than one round of the scan over them."""
    rng = np.random.default_rng(3)
    run([1] * 700, rng.integers(0, 90, size=700).tolist(), "star", 2, 1, 64, "bf16", 16)
    sizes = rng.integers(0, 4, size=300)
    sizes[0] = 3
    run(sizes.tolist(), rng.integers(0, 50, size=300).tolist(), "chain", 2, 1, 64, "f32", 8, ragged=True)


@pytest.mark.parametrize("n,hq,hkv,d", [(128, 8, 2, 128), (70, 8, 1, 64), (33, 4, 1, 256)])
def test_dense_blocks_side_by_side(n, hq, hkv, d):
    """Blocks of rows that share keys, contexts of different lengths."""
    run([n] * 3, [1000, 37, 511], "rrt", hq, hkv, d, "bf16", 32)


def test_large_scores():
    """Scores of some hundreds: one key has all the weight, the running maximum moves often."""
    run([12, 12], [300, 90], "rrt", 4, 2, 64, "bf16", 16, qstd=60.0)
    run([12, 12], [300, 90], "rrt", 4, 2, 64, "f32", 16, qstd=60.0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq", [(6, 2), (40, 2), (70, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite(io, n, hq, bad):
    """A node's value that is not finite reaches the node and its descendants and nobody else."""
    c = Case([n, n], [33, 0], "rrt", hq, 2, 64, io, 16)
    for node, col in ((2, 5), (n - 1, 63)):
        c.fused[n + node, hq + 2, col] = bad
        c.fused64[n + node, hq + 2, col] = bad
    o = c.call()
    c.check(o)


def test_keys_that_are_not_finite():
    """A node's key of NaN makes the node and its descendants NaN and nobody else."""
    c = Case([9], [20], "rrt", 2, 2, 64, "bf16", 16)
    c.fused[3, 2] = float("nan")
    o = c.call().float().cpu().numpy()
    sees = c.anc[0][:, 3] | (np.arange(9) == 3)
    assert np.array_equal(np.isnan(o[:, 0]).all(-1), sees) and not np.isnan(o[:, 1]).any()


def test_invalid_sequences_are_nan():
    """A failed tree, a length outside the table and a page outside the pool: NaN rows, and the
    other sequences as they are."""
    c = Case([4] * 6, [50, 50, 50, 50, 50, 50], "chain", 4, 2, 64, "bf16", 16)
    c.status[1] = 3
    c.ctx_dev[2] = -1
    c.ctx_dev[3] = 16 * c.table.shape[1] + 1
    c.table_dev[4, 1] = c.pools[0].shape[0]
    c.table_dev[5, 3] = -1
    o = c.call()
    c.check(o, skip=(1, 2, 3, 4, 5))
    assert torch.isnan(o[4:24]).all()


def test_rows_that_belong_to_nobody_stay():
    c = Case([3, 4], [20, 10], "chain", 2, 1, 64, "bf16", 16, ragged=True, N=4)
    wide = torch.full((c.rows + 2, c.hq, c.d), 7.0, dtype=c.fused.dtype, device="cuda")
    extra = torch.cat([c.fused, c.fused[:2]])
    hq, hkv = c.hq, c.hkv
    T.gdn_attn_verify(c.dims, c.cache, c.table_dev, c.ctx_dev, extra[:, :hq], extra[:, hq:hq + hkv],
                      extra[:, hq + hkv:], c.anc_dev, c.status, wide, c.ws, offsets=c.off_dev)
    c.check(wide[:c.rows])
    assert (wide[c.rows:] == 7.0).all()


def test_unusable_offsets():
    """A sequence of more rows than N is not touched; the others are as they are."""
    c = Case([3, 4], [20, 10], "chain", 2, 1, 64, "bf16", 16, ragged=True, N=4)
    c.off_dev[1] = 8                             # 8 rows of at most 4, then a negative count
    o = c.call()
    assert (o == 7.0).all()


def test_padding_bits_are_not_nodes():
    c = Case([3, 4], [20, 10], "chain", 2, 1, 64, "bf16", 16, ragged=True, N=40)
    c.anc_dev[0, :, 0] |= ~7
    c.anc_dev[:, :, 1] = -1
    c.check(c.call())


def test_other_stream_and_graph():
    """On a stream of its own, and captured: every replay gives the eager bits, with eager work
    between the replays."""
    c = Case([20] * 3, [400, 10, 77], "rrt", 4, 2, 128, "bf16", 16)
    want = c.call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = torch.zeros_like(want)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.call(o)
    s.synchronize()
    assert torch.equal(o, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(o)
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        assert torch.equal(c.call(), want)


def test_layers():
    """A layer of a pool of several."""
    c = Case([5], [40], "rrt", 2, 1, 64, "bf16", 16)
    k5 = torch.stack([torch.full_like(c.pools[0], float("nan")), c.pools[0], torch.zeros_like(c.pools[0])])
    v5 = torch.stack([torch.zeros_like(c.pools[1]), c.pools[1], torch.full_like(c.pools[1], float("nan"))])
    o = torch.empty((c.rows, c.hq, c.d), dtype=c.fused.dtype, device="cuda")
    T.gdn_attn_verify(c.dims, T.PagedCache(k5, v5), c.table_dev, c.ctx_dev, c.fused[:, :2], c.fused[:, 2:3],
                      c.fused[:, 3:], c.anc_dev, c.status, o, c.ws, layer=1)
    c.check(o)
