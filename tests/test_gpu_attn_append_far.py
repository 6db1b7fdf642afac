"""Append where a sequence's length reaches the last that 32 bits hold."""
import pytest
import torch

from test_gpu_attn_pages import DEV, i32

pytestmark = pytest.mark.gpu
T = pytest.importorskip("tree_masked_gated_amd")


def test_append_at_the_longest_length():
    """Three sequences of 2^31 - 3 rows: two more rows have a place, three have not, and nothing of
    them is appended."""
    page, width, d = 65536, 32768, 8
    table = torch.arange(3, dtype=torch.int32, device=DEV)[:, None].repeat(1, width).contiguous()
    kp = torch.zeros(3, page, 1, d, device=DEV)
    vp = torch.zeros_like(kp)
    x = torch.ones(3 * 3, 2, d, device=DEV)
    new_len = torch.empty(3, dtype=torch.int32, device=DEV)
    T.gdn_attn_commit(T.attn_dims(3, 3, 1, 1, d, "f32"), T.PagedCache(kp, vp), table, i32([2 ** 31 - 3] * 3), x[:, :1],
                      x[:, 1:], i32([[0, 1, 2]] * 3), i32([2, 3, 0]), new_len)
    assert new_len.tolist() == [2 ** 31 - 1, -1, 2 ** 31 - 3]
    for pool in (kp, vp):
        assert pool[0, page - 3:page - 1].eq(1).all() and pool[0].sum() == 2 * d
        assert pool[1:].abs().sum() == 0
