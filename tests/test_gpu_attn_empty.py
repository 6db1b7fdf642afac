"""Batches in which nothing is cached yet (a table without columns) and batches of trees without nodes."""
import pytest
import torch

from test_gpu_attn_pages import DEV, i32
from test_gpu_attn_verify import Case

pytestmark = pytest.mark.gpu
T = pytest.importorskip("tree_masked_gated_amd")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq", [(1, 2), (9, 4), (90, 8)])
def test_verify_without_a_prefix(io, n, hq):
    """No sequence has a prefix, and the table no columns."""
    c = Case([n] * 3, [0, 0, 0], "rrt", hq, 2, 64, io, 16)
    c.table_dev = c.table_dev[:, :0].contiguous()
    c.check(c.call())
    c.ctx_dev[1] = 1                             # a row that no page holds
    o = c.call()
    c.check(o, skip=(1,))
    assert torch.isnan(o[n:2 * n]).all()


def test_commit_without_a_table():
    """No row has a place; a path of nothing asks for none."""
    kp = torch.zeros(2, 4, 1, 8, device=DEV)
    x = torch.ones(2 * 3, 2, 8, device=DEV)
    new_len = torch.empty(2, dtype=torch.int32, device=DEV)
    T.gdn_attn_commit(T.attn_dims(2, 3, 1, 1, 8, "f32"), T.PagedCache(kp, kp.clone()), i32([[], []]), i32([0, 0]),
                      x[:, :1], x[:, 1:], i32([[0, 1, 2]] * 2), i32([0, 1]), new_len)
    assert new_len.tolist() == [0, -1] and kp.abs().sum() == 0


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_trees_without_nodes(io):
    """Ragged calls of no rows at all: nothing to rotate and to attend, lengths stay."""
    B, d = 3, 64
    dims = T.attn_dims(B, 8, 4, 2, d, "f32" if io == torch.float32 else "bf16")
    kp = torch.ones(4, 16, 2, d, device=DEV, dtype=io)
    cache = T.PagedCache(kp, kp.clone())
    off, table, ctx = i32([0] * (B + 1)), i32([[0], [1], [2]]), i32([5, 0, 16])
    q, k = (torch.empty(0, h, d, device=DEV, dtype=io) for h in (4, 2))
    T.gdn_attn_rope(dims, T.rope_dims(d), q, k, torch.ones(d // 2, dtype=torch.float64, device=DEV), ctx,
                    i32([[0] * 8] * B), q, k, offsets=off)
    T.gdn_attn_verify(dims, cache, table, ctx, q, k, k, i32([[[0]] * 8] * B), i32([0] * B), q, T.attn_workspace(dims),
                      offsets=off)
    new_len = torch.empty(B, dtype=torch.int32, device=DEV)
    T.gdn_attn_commit(dims, cache, table, ctx, k, k, i32([]), i32([0, -1, 1]), new_len, offsets=off)
    assert new_len.tolist() == [5, 0, -1] and kp.eq(1).all()
