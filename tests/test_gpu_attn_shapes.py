"""Tree attention in the shapes that full batches take: enough blocks of rows that the kernel uses its
tiles of 128 and 256 rows, against the same 64-bit reference and bounds as test_gpu_attn_verify."""
import numpy as np
import pytest

from test_gpu_attn_verify import Case, run

pytestmark = pytest.mark.gpu


def lengths(batch, most, seed):
    """Contexts around the tiles' edges, most of them short."""
    rng = np.random.default_rng(seed)
    c = rng.choice([0, 1, 15, 63, 64, 65, 127, 128, 130, 191, 192, 193, 256], size=batch)
    c[:4] = (most, 0, most - 1, 64)
    return c.tolist()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 24, 5])
@pytest.mark.parametrize("ragged", [False, True])
def test_rows_256(d, page, ragged):
    """160 rows of a key head: one block of 256 to each of 132."""
    sizes = [40] * 33 if not ragged else [40, 1, 0, 39] + [33, 40, 17] * 9 + [40, 36]
    run(sizes, lengths(33, 520, page), "rrt", 16, 4, d, "bf16", page, ragged=ragged)


@pytest.mark.parametrize("d", [72, 120])
def test_rows_256_padded_head(d):
    """Head sizes that leave columns of the tile unused, over pages with NaN in rows that nobody owns."""
    run([40] * 33, lengths(33, 300, d), "rrt", 16, 4, d, "bf16", 16, order="heads")


@pytest.mark.parametrize("n,hq,hkv", [(130, 8, 4), (100, 20, 4)])
def test_blocks_of_256_side_by_side(n, hq, hkv):
    """Several blocks of 256 rows over the same keys, the last one partly filled."""
    run([n] * 18, lengths(18, 400, n), "rrt", hq, hkv, 64, "bf16", 32)


@pytest.mark.parametrize("d", [64, 128, 104])
@pytest.mark.parametrize("page", [16, 7])
def test_rows_128(d, page):
    """100 rows of a key head: blocks of 128."""
    run([25] * 33, lengths(33, 520, d + page), "chain", 16, 4, d, "bf16", page)


@pytest.mark.parametrize("d", [136, 256])
def test_rows_128_wide_head(d):
    run([25] * 33, lengths(33, 200, d), "rrt", 16, 4, d, "bf16", 16)


def test_large_scores_in_blocks():
    """The running maximum moves often while the next tile's scores are formed ahead."""
    run([40] * 33, lengths(33, 520, 1), "rrt", 16, 4, 64, "bf16", 16, qstd=60.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_in_blocks(bad):
    """In a block that several workgroups share, and in one of a single workgroup."""
    c = Case([40] * 33, lengths(33, 520, 2), "rrt", 16, 4, 64, "bf16", 16)
    for b, node, col in ((0, 3, 5), (1, 39, 63), (2, 20, 0)):
        row = 40 * b + node
        c.fused[row, 16 + 4 + 1, col] = bad
        c.fused64[row, 16 + 4 + 1, col] = bad
    c.check(c.call())


def test_invalid_sequences_in_blocks():
    """A page outside the pool in a context that several workgroups share: NaN rows, the others as
    they are."""
    import torch
    c = Case([40] * 33, lengths(33, 520, 4), "rrt", 16, 4, 64, "bf16", 16)
    c.table_dev[0, 7] = c.pools[0].shape[0]
    c.status[3] = 2
    o = c.call()
    c.check(o, skip=(0, 3))
    assert torch.isnan(o[:40]).all() and torch.isnan(o[120:160]).all()


@pytest.mark.parametrize("n,hq", [(9, 2), (40, 8), (70, 8)])
def test_one_sequence_in_many_parts(n, hq):
    """Few blocks of rows and many keys: each block is joined from many workgroups' parts."""
    run([n], [9000], "rrt", hq, 2, 128, "bf16", 16)
