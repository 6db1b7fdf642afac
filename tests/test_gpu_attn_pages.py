"""Append and page bookkeeping against plain Python, whole numbers and copied rows equal."""
import numpy as np
import pytest
import torch

import page_reference as R

pytestmark = pytest.mark.gpu
T = pytest.importorskip("tree_masked_gated_amd")
DEV = "cuda"


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def pool(rng, shape, io, order):
    t = torch.from_numpy(rng.standard_normal(shape)).to(torch.float32 if io == "f32" else torch.bfloat16).to(DEV)
    return t.transpose(-3, -2).contiguous().transpose(-3, -2) if order == "heads" else t


# ------------------------------------------------------------------ append

def append(sizes, N, ctx, taken, hkv, d, io, page, order="rows", ragged=False, seed=0, spoil=None):
    """spoil(table, path): changes before the call; sequences it makes unusable are returned by it."""
    print("[gpu-append]", sizes, ctx, taken, hkv, d, io, page, order, flush=True)
    rng = np.random.default_rng(seed)
    B, rows = len(sizes), sum(sizes)
    width = max(-(-(c + n) // page) for c, n in zip(ctx, sizes)) + 1
    n_pages = B * width + 2
    table = rng.permutation(n_pages)[:B * width].reshape(B, width)
    kp, vp = (pool(rng, (n_pages, page, hkv, d), io, order) for _ in range(2))
    fused = torch.from_numpy(rng.standard_normal((rows, 2 * hkv, d))).to(kp.dtype).to(DEV)
    off = np.concatenate([[0], np.cumsum(sizes)])
    path = np.full(rows, -1)
    for b in range(B):
        path[off[b]:off[b] + max(taken[b], 0)] = np.sort(rng.permutation(sizes[b])[:max(taken[b], 0)])
    wrong = spoil(table, path) if spoil else ()
    new_len = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    want_k, want_v, want_len = kp.clone(), vp.clone(), []
    for b in range(B):
        m = max(taken[b], 0)
        want_len.append(-1 if b in wrong else ctx[b] + m)
        if b in wrong:
            continue
        for t in range(m):
            at = (int(table[b, (ctx[b] + t) // page]), (ctx[b] + t) % page)
            want_k[at], want_v[at] = fused[off[b] + path[off[b] + t], :hkv], fused[off[b] + path[off[b] + t], hkv:]
    T.gdn_attn_commit(T.attn_dims(B, N, hkv, hkv, d, io), T.PagedCache(kp, vp), i32(table), i32(ctx),
                      fused[:, :hkv], fused[:, hkv:], i32(path if ragged else path.reshape(B, N)), i32(taken), new_len,
                      offsets=i32(off) if ragged else None)
    assert new_len.tolist() == want_len
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["rows", "heads"])
@pytest.mark.parametrize("page,d,hkv", [(1, 8, 1), (16, 128, 4), (24, 72, 3)])
def test_append(io, order, page, d, hkv):
    append([20] * 5, 20, [0, 5, 47, 48, 100], [20, 0, 3, 1, 17], hkv, d, io, page, order)


def test_append_ragged_and_long():
    append([0, 7, 1, 40], 40, [3, 16, 0, 9], [0, 7, 1, 33], 2, 64, "bf16", 16, ragged=True)
    append([1024], 1024, [5], [1024], 2, 128, "f32", 16)
    append([3, 3], 3, [10, 10], [-1, 2], 1, 64, "bf16", 16)            # an invalid tree's path


def test_append_refuses_whole_sequences():
    def spoil(table, path):
        table[1, 1] = 10 ** 6                   # no such page, in the middle of the path
        table[2, 0] = -1                        # not needed: the path begins in page 1
        path[3 * 6 + 2] = 6                     # no such node
        return (1, 3)
    append([6] * 5, 6, [2, 2, 4, 2, 2], [6, 6, 6, 6, 0], 2, 64, "bf16", 4, spoil=spoil)


def test_append_past_the_table():
    kp = torch.zeros(4, 4, 1, 8, device=DEV)
    x = torch.ones(3 * 3, 2, 8, device=DEV)
    new_len = torch.empty(3, dtype=torch.int32, device=DEV)
    T.gdn_attn_commit(T.attn_dims(3, 3, 1, 1, 8, "f32"), T.PagedCache(kp, kp.clone()), i32([[0], [1], [2]]),
                      i32([2, 1, -1]), x[:, :1], x[:, 1:], i32([[0, 1, 2]] * 3), i32([3, 3, 1]), new_len)
    assert new_len.tolist() == [-1, 4, -1]
    assert kp[0].sum() == 0 and kp[1].sum() == 24 and kp[2].sum() == 0


# ------------------------------------------------------------------ bookkeeping

class Pool:
    def __init__(self, rng, n_pages, page, slots, width, fill, share=0.0):
        """Random sequences; with probability `share` one shares a run of pages with an earlier one."""
        self.page, self.width = page, width
        self.ref = [0] * n_pages
        self.table = [[-1] * width for _ in range(slots)]
        self.held, self.length = [0] * slots, [0] * slots
        ids = rng.permutation(n_pages).tolist()
        for s in range(slots):
            if rng.random() > fill:
                continue
            other = int(rng.integers(0, s)) if s else 0
            if rng.random() < share and self.held[other]:
                n = int(rng.integers(1, self.held[other] + 1))
                mine = self.table[other][:n]
            else:
                n = int(rng.integers(0, width + 1))
                if n > len(ids):
                    continue
                mine = [ids.pop() for _ in range(n)]
            for p in mine:
                self.ref[p] += 1
            self.table[s][:n] = mine
            self.held[s] = n
            self.length[s] = int(rng.integers(max(0, (n - 2) * page), n * page + 1)) if n else 0
        self.dims = T.page_dims(n_pages, page, slots, width)

    def device(self):
        return [i32(self.ref), i32(self.table), i32(self.held), i32(self.length)]

    def host(self):
        return self.ref, self.table, self.held, self.length

    def check(self, dev):
        for got, want in zip(dev, self.host()):
            assert np.array_equal(got.cpu().numpy(), np.array(want, dtype=np.int32))


SHAPES = [(1, 1, 1, 1), (9, 4, 3, 3), (100, 16, 20, 8), (5000, 16, 300, 40), (20000, 32, 4096, 6)]


@pytest.mark.parametrize("n_pages,page,slots,width", SHAPES)
@pytest.mark.parametrize("seed", range(3))
def test_fork(n_pages, page, slots, width, seed):
    rng = np.random.default_rng(seed)
    p = Pool(rng, n_pages, page, slots, width, 0.5)
    n = max(1, slots // 2)
    src, dst = rng.integers(-1, slots + 1, size=n), rng.integers(-1, slots + 1, size=n)
    dev, status = p.device(), torch.full((n,), 9, dtype=torch.int32, device=DEV)
    T.gdn_pages_fork(p.dims, i32(src), i32(dst), *dev, status)
    assert status.tolist() == R.fork(page, width, src.tolist(), dst.tolist(), *p.host())
    p.check(dev)


@pytest.mark.parametrize("n_pages,page,slots,width", SHAPES)
@pytest.mark.parametrize("seed", range(4))
def test_reserve(n_pages, page, slots, width, seed):
    """Plenty of pages, too few, shared last pages that all or some of their holders ask for."""
    rng = np.random.default_rng(seed)
    p = Pool(rng, n_pages, page, slots, width, [0.3, 0.9, 0.6, 1.0][seed], 0.6)
    need = rng.integers(-2, 2 * page + 1, size=slots) * (rng.random(slots) < [0.3, 0.9, 1.0, 1.0][seed])
    dev = p.device()
    src, dst, status = (torch.full((slots,), 9, dtype=torch.int32, device=DEV) for _ in range(3))
    count = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    T.gdn_pages_reserve(p.dims, i32(need), *dev, src, dst, count, status)
    want, moves = R.reserve(page, width, need.tolist(), *p.host())
    assert status.tolist() == want
    n = int(count)
    assert list(zip(src[:n].tolist(), dst[:n].tolist())) == moves
    p.check(dev)


def test_reserve_contradictions():
    """A length past the held pages, a last page that is none: refused, nothing changed."""
    p = Pool(np.random.default_rng(0), 8, 4, 3, 4, 0.0)
    p.length, p.held = [5, 5, 0], [1, 2, 0]
    p.table[0][0], p.table[1][:2], p.ref = 0, [1, 77], [1, 1, 0, 0, 0, 0, 0, 0]
    dev = p.device()
    s, d, st = (torch.zeros(3, dtype=torch.int32, device=DEV) for _ in range(3))
    c = torch.zeros(1, dtype=torch.int32, device=DEV)
    T.gdn_pages_reserve(p.dims, i32([1, 1, 9]), *dev, s, d, c, st)
    assert st.tolist() == [-1, -1, 0] and int(c) == 0
    assert dev[2].tolist() == [1, 2, 3] and dev[1][2].tolist() == [2, 3, 4, -1]


@pytest.mark.parametrize("n_pages,page,slots,width", SHAPES)
def test_free(n_pages, page, slots, width):
    rng = np.random.default_rng(1)
    p = Pool(rng, n_pages, page, slots, width, 0.8, 0.4)
    drop = rng.integers(0, 2, size=slots)
    dev = p.device()
    T.gdn_pages_free(p.dims, i32(drop), *dev)
    R.free(drop.tolist(), *p.host())
    p.check(dev)


@pytest.mark.parametrize("n_pages,page,slots,width", SHAPES)
@pytest.mark.parametrize("most", [1, 7, 100000])
def test_compact(n_pages, page, slots, width, most):
    rng = np.random.default_rng(2)
    p = Pool(rng, n_pages, page, slots, width, 0.7, 0.2)
    dev = p.device()
    src, dst = (torch.full((most,), 9, dtype=torch.int32, device=DEV) for _ in range(2))
    count, remap = torch.empty(1, dtype=torch.int32, device=DEV), torch.empty(n_pages, dtype=torch.int32, device=DEV)
    T.gdn_pages_compact(p.dims, dev[0], dev[1], dev[2], src, dst, count, remap)
    moves, where = R.compact(most, p.ref, p.table)
    n = int(count)
    assert list(zip(src[:n].tolist(), dst[:n].tolist())) == moves
    assert remap.tolist() == where
    p.check(dev)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("layers,page,hkv,d", [(1, 1, 1, 8), (3, 16, 4, 128), (2, 24, 3, 72), (1, 1000, 2, 64)])
@pytest.mark.parametrize("order", ["rows", "heads", "loose"])
def test_copy(io, layers, page, hkv, d, order):
    """Dense pages in both orders, and pages whose rows lie apart."""
    rng = np.random.default_rng(4)
    n_pages = 12
    if order == "loose":
        big = pool(rng, (2, layers, n_pages, page + 1, hkv + 1, d + 8), io, "rows")
        kp, vp = (x[..., :page, :hkv, :d] for x in big)
    else:
        kp, vp = (pool(rng, (layers, n_pages, page, hkv, d), io, order) for _ in range(2))
    src, dst = [3, 5, 3, 9, 40, 1], [0, 11, 7, -1, 2, 4]
    want = []
    for x in (kp, vp):
        w = x.clone()
        for s, t in list(zip(src, dst))[:5]:
            if 0 <= s < n_pages and 0 <= t < n_pages:
                w[:, t] = x[:, s]
        want.append(w)
    T.gdn_pages_copy(T.PagedCache(kp, vp), i32(src), i32(dst), i32([5]))
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    T.gdn_pages_copy(T.PagedCache(kp, vp), i32(src), i32(dst), i32([0]))
    assert torch.equal(kp, want[0])


def test_pages_in_a_graph():
    """Reserve, copy and free captured: every replay on restored state gives the eager result."""
    rng = np.random.default_rng(6)
    p = Pool(rng, 400, 16, 30, 10, 0.7, 0.6)
    need = i32(rng.integers(0, 20, size=30))
    drop = i32(rng.integers(0, 2, size=30))
    kp, vp = (pool(rng, (1, 400, 16, 1, 8), "f32", "rows") for _ in range(2))
    cache = T.PagedCache(kp, vp)
    start = p.device() + [kp.clone(), vp.clone()]
    state = [x.clone() for x in start[:4]] + [kp, vp]
    src, dst, status = (torch.zeros(30, dtype=torch.int32, device=DEV) for _ in range(3))
    count = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        T.gdn_pages_reserve(p.dims, need, *state[:4], src, dst, count, status)
        T.gdn_pages_copy(cache, src, dst, count)
        T.gdn_pages_free(p.dims, drop, *state[:4])

    def restore():
        for x, y in zip(state, start):
            x.copy_(y)

    step()
    want = [x.clone() for x in state]
    restore()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        restore()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(state, want))
