"""Sizes that would overflow the kernels' 32-bit counts are refused on the host.  CPU only: every call
here ends before a launch."""
import ctypes

import pytest

from test_attn_abi import FAKE, NO_GPU, cache, dims, rows

T = pytest.importorskip("tree_masked_gated_amd")
DIMS, NULL = -2, -1


def ref(x):
    return ctypes.byref(x)


def rope(d):
    """No freq: the sizes are checked before."""
    r = rows()
    return T._lib.gdn_attn_rope(ref(d), ref(T.RopeDims(32, 0, 1.0)), None, 6, ref(r), ref(r), None, FAKE, FAKE, ref(r),
                                ref(r), None)


def commit(d, c):
    """No path: the sizes are checked before."""
    r = rows()
    return T._lib.gdn_attn_commit(ref(d), None, ref(c), 0, FAKE, 4, FAKE, ref(r), ref(r), None, FAKE, FAKE + 64, None)


def verify(d, c):
    """An odd workspace: refused where the sizes are not."""
    r = rows()
    return T._lib.gdn_attn_verify(ref(d), None, ref(c), 0, FAKE, 4, FAKE, ref(r), ref(r), ref(r), FAKE, FAKE, ref(r),
                                  None, None)


@NO_GPU
@pytest.mark.parametrize("hq,hkv,rc", [(2 ** 20, 2 ** 13, NULL), (2 ** 16, 1, NULL), (2 ** 20 + 2 ** 13, 2 ** 13, DIMS),
                                       (2 ** 13 + 1, 2 ** 13 + 1, DIMS), (2 ** 30, 2 ** 30, DIMS),
                                       (2 ** 31 - 1, 2 ** 31 - 1, DIMS)])
def test_heads(hq, hkv, rc):
    d = dims(n_nodes=1, h_q=hq, h_kv=hkv)
    assert rope(d) == rc
    assert commit(d, cache(h_kv=hkv, page_rows=1)) == rc
    assert verify(d, cache(h_kv=hkv, page_rows=1)) == rc


@NO_GPU
@pytest.mark.parametrize("page_rows,hkv,d,io,rc", [(65536, 256, 256, 0, NULL), (65536, 257, 256, 0, DIMS),
                                                   (65536, 2 ** 31 - 1, 8, 1, DIMS), (65536, 8192, 32, 1, DIMS),
                                                   (65536, 8192, 16, 1, NULL)])
def test_page_bytes(page_rows, hkv, d, io, rc):
    c = cache(page_rows=page_rows, h_kv=hkv, d=d, io_dtype=io)
    assert T._lib.gdn_pages_copy(ref(c), 2, FAKE, FAKE, None, None) == rc


@NO_GPU
@pytest.mark.parametrize("name", ["k_page", "v_page", "k_row", "v_row"])
def test_strides_in_pieces_of_16_bytes(name):
    """Offsets in a pool are products of 32-bit page ids and row numbers with 32-bit strides in pieces."""
    for elements, rc in ((4 * (2 ** 32 - 1), NULL), (4 * 2 ** 32, DIMS), (2 ** 61, DIMS), (2 ** 62, DIMS),
                         (2 ** 63 - 4, DIMS)):
        c = cache(**{name: elements})
        r = rows()
        got = T._lib.gdn_attn_verify(ref(dims()), None, ref(c), 0, FAKE, 4, FAKE, ref(r), ref(r), ref(r), FAKE, FAKE,
                                     ref(r), FAKE, None) if rc == DIMS else verify(dims(), c)
        assert got == rc, elements
