"""Pools and row tensors whose offsets pass 2^32 bytes."""
import numpy as np
import pytest
import torch

from test_gpu_attn_pages import DEV, i32
from test_gpu_attn_verify import Case

pytestmark = pytest.mark.gpu
T = pytest.importorskip("tree_masked_gated_amd")

FAR = 5 << 30                                    # bytes


def far_pool(near, ids):
    """A pool of FAR bytes of the near one's page shape, with the near one's pages at `ids`."""
    n = FAR // (near[0].numel() * near.element_size())
    x = torch.empty((n, *near.shape[1:]), dtype=near.dtype, device=DEV)
    x[ids] = near
    return x


def last_ids(near):
    """Pages beyond 2^32 bytes, in descending order."""
    n = FAR // (near[0].numel() * near.element_size())
    return torch.arange(n - 1, n - 1 - len(near), -1, device=DEV)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq", [(1, 8), (20, 4), (60, 8)])
def test_verify_far_pages(io, n, hq):
    """Every page lies past 2^32 bytes: the same bits as from a small pool."""
    print("[gpu-attn-far]", io, n, hq, flush=True)
    c = Case([n] * 2, [700, 65], "rrt", hq, 2, 128, io, 16)
    want = c.call()
    c.check(want)
    ids = last_ids(c.pools[0])
    c.cache = T.PagedCache(*(far_pool(p, ids) for p in c.pools))
    held = c.table_dev >= 0
    c.table_dev[held] = ids[c.table_dev[held].long()].int()
    assert torch.equal(c.call().view(torch.uint8), want.view(torch.uint8))


def test_append_and_copy_far_pages():
    """Rows and pages written past 2^32 bytes, and none of the pages before them."""
    near = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16, device=DEV)
    ids = last_ids(near)
    kp, vp = far_pool(near, ids), far_pool(near, ids)
    wrapped = (ids * near[0].numel() * 2 % (1 << 32)) // (near[0].numel() * 2)       # where 32 bits would lead
    for p in (kp, vp):
        p[wrapped] = 3
    x = torch.randn(6, 16, 128, device=DEV).bfloat16()
    new_len = torch.empty(1, dtype=torch.int32, device=DEV)
    T.gdn_attn_commit(T.attn_dims(1, 6, 8, 8, 128, "bf16"), T.PagedCache(kp, vp), ids[None, :2].int().contiguous(), i32([14]),
                      x[:, :8], x[:, 8:], i32([[0, 2, 3, 5, -1, -1]]), i32([4]), new_len)
    assert new_len.tolist() == [18]
    for p, y in ((kp, x[:, :8]), (vp, x[:, 8:])):
        assert torch.equal(p[ids[0], 14:], y[[0, 2]]) and torch.equal(p[ids[1], :2], y[[3, 5]])
        assert p[ids[0], :14].eq(0).all() and p[ids[1], 2:].eq(0).all()
    T.gdn_pages_copy(T.PagedCache(kp, vp), ids[:2].int().contiguous(), ids[2:].int().contiguous(), i32([2]))
    for p in (kp, vp):
        assert torch.equal(p[ids[2:]], p[ids[:2]]) and p[wrapped].eq(3).all()


def test_rows_far_apart():
    """Rows of q, k, v and o with 2^28 elements between them: rotated and attended as from dense tensors."""
    rows, step = 20, 1 << 28
    c = Case([rows], [50], "rrt", 4, 2, 64, "bf16", 16)
    want = c.call()
    c.check(want)
    buf = torch.empty((rows - 1) * step + 1024, dtype=torch.bfloat16, device=DEV)
    far = buf.as_strided((rows, 12, 64), (step, 64, 1))          # q, k, v, o
    far[:, :8] = c.fused
    o = far[:, 8:]
    T.gdn_attn_verify(c.dims, c.cache, c.table_dev, c.ctx_dev, far[:, :4], far[:, 4:6], far[:, 6:8], c.anc_dev, c.status, o,
                      c.ws)
    assert torch.equal(o, want)
    freq = torch.from_numpy(10000.0 ** (-np.arange(0, 64, 2) / 64)).to(DEV)
    depth = torch.arange(rows, dtype=torch.int32, device=DEV)[None]
    q, k = c.fused[:, :4].contiguous(), c.fused[:, 4:6].contiguous()
    T.gdn_attn_rope(c.dims, T.rope_dims(64), q, k, freq, c.ctx_dev, depth, q, k)
    T.gdn_attn_rope(c.dims, T.rope_dims(64), far[:, :4], far[:, 4:6], freq, c.ctx_dev, depth, far[:, :4], far[:, 4:6])
    assert torch.equal(far[:, :4], q) and torch.equal(far[:, 4:6], k)
    new_len = torch.empty(1, dtype=torch.int32, device=DEV)
    kp, vp = (torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    T.gdn_attn_commit(c.dims, T.PagedCache(kp, vp), i32([[1, 0]]), i32([15]), far[:, 4:6], far[:, 6:8],
                      i32([[0, 17, 19] + [-1] * 17]), i32([3]), new_len)
    assert new_len.tolist() == [18]
    for p, y in ((kp, far[:, 4:6]), (vp, far[:, 6:8])):
        assert torch.equal(p[1, 15], y[0]) and torch.equal(p[0, :2], y[[17, 19]])
