"""Reservation of pages at the numbers of slots where the kernel's table of shared pages grows: its LDS, static and
dynamic together, passes 64 KiB between 512 and 1024 slots."""
import numpy as np
import pytest
import torch

import page_reference as R
from test_gpu_attn_pages import DEV, Pool, i32

pytestmark = pytest.mark.gpu
T = pytest.importorskip("tree_masked_gated_amd")


@pytest.mark.parametrize("slots", [1, 32, 33, 256, 257, 512, 513, 1000, 1024, 1025, 2048, 2049, 4096])
def test_reserve_slots(slots):
    print("[gpu-reserve]", slots, flush=True)
    rng = np.random.default_rng(slots)
    page, width, n_pages = 16, 5, 3 * slots + 7
    p = Pool(rng, n_pages, page, slots, width, 0.8, 0.6)
    need = rng.integers(-2, 2 * page + 1, size=slots)
    dev = p.device()
    src, dst, status = (torch.full((slots,), 9, dtype=torch.int32, device=DEV) for _ in range(3))
    count = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    T.gdn_pages_reserve(p.dims, i32(need), *dev, src, dst, count, status)
    want, moves = R.reserve(page, width, need.tolist(), *p.host())
    assert status.tolist() == want
    n = int(count)
    assert list(zip(src[:n].tolist(), dst[:n].tolist())) == moves
    p.check(dev)
