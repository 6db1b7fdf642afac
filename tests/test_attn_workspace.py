"""Sizes of the tree attention's workspace.  CPU only."""
import itertools

import pytest

T = pytest.importorskip("tree_masked_gated_amd")


def need(batch, nodes, hq, hkv, d, io):
    return T.gdn_attn_workspace_bytes(T.attn_dims(batch, nodes, hq, hkv, d, io))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_counters_do_not_depend_on_the_batch(io):
    """Partial results begin at one place for every batch: a call of another batch on the same workspace
    does not write over the arrival counters."""
    for d in (64, 128, 256):
        assert len({need(b, 1, 8, 8, d, io) for b in (1, 8, 32, 64, 1000)}) == 1
        assert len({need(b, 1, 8 * h, h, d, io) for b in (1, 64) for h in (1, 2, 8)}) == 1


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 64, 72, 128, 136, 256])
def test_fewer_sequences_and_nodes_need_no_more(io, d):
    batches, nodes = (1, 2, 7, 16, 33, 64, 128, 1000), (1, 2, 5, 16, 17, 33, 64, 65, 129, 300, 1024)
    for hq, hkv in ((1, 1), (8, 1), (16, 4), (32, 4)):
        size = {(b, n): need(b, n, hq, hkv, d, io) for b, n in itertools.product(batches, nodes)}
        for (b, n), (c, m) in itertools.product(size, size):
            if b <= c and n <= m:
                assert size[b, n] <= size[c, m], (hq, hkv, b, n, c, m)
