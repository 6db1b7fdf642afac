"""The attention calls' symbols, struct layouts and host-side refusals.  CPU only: no call here
reaches a kernel launch."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from attn_reference import ancestors, attend, pack_bits, parents
import page_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_attn.h")

T = pytest.importorskip("tree_masked_gated_amd")
NO_GPU = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                            reason="fake device pointers are only passed where no GPU exists")
FAKE, ODD = 0x10000, 0x10004


def test_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\bint (gdn_\w+)\s*\(", src)))
    assert names == ["gdn_attn_commit", "gdn_attn_rope", "gdn_attn_verify", "gdn_attn_workspace_bytes",
                     "gdn_pages_compact", "gdn_pages_copy", "gdn_pages_fork", "gdn_pages_free", "gdn_pages_reserve"]
    out = subprocess.run(["nm", "-D", "--defined-only", T.lib_path], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\sT\s(\w+)", out))
    assert set(names) <= exported
    assert all(n in T.__all__ for n in names)


def test_header_compiles_as_c_and_structs_match():
    """The header is plain C, and the binding's structs have the compiler's sizes and offsets."""
    pairs = [("gdn_attn_dims", T.AttnDims), ("gdn_rope_dims", T.RopeDims), ("gdn_page_dims", T.PageDims),
             ("gdn_attn_rows", T.AttnRows), ("gdn_paged_cache", T.PagedCacheStruct)]
    lines = ["#include <stddef.h>", '#include "gdn_attn.h"']
    for c, py in pairs:
        lines.append(f"_Static_assert(sizeof({c}) == {ctypes.sizeof(py)}, \"{c}\");")
        for f, _ in py._fields_:
            lines.append(f"_Static_assert(offsetof({c}, {f}) == {getattr(py, f).offset}, \"{c}.{f}\");")
    p = subprocess.run(["gcc", "-x", "c", "-std=c11", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), "-I",
                        "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-"], input="\n".join(lines) + "\n", text=True,
                       capture_output=True)
    assert p.returncode == 0, p.stderr


def rows(data=FAKE, row=64, head=32):
    return T.AttnRows(data, row, head)


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, n_layers=1, n_pages=4, page_rows=16, h_kv=2, d=32, io_dtype=0, k_layer=0, k_page=1024,
             k_row=64, k_head=32, v_layer=0, v_page=1024, v_row=64, v_head=32)
    f.update(kw)
    return T.PagedCacheStruct(**f)


def dims(**kw):
    f = dict(batch=2, n_nodes=3, h_q=4, h_kv=2, d=32, io_dtype=0, scale=0.2)
    f.update(kw)
    return T.AttnDims(**f)


BAD_DIMS = [(dict(batch=-1), -2), (dict(n_nodes=0), -2), (dict(n_nodes=1025), -2), (dict(h_q=3), -2),
            (dict(h_q=0), -2), (dict(h_kv=0), -2), (dict(d=0), -2), (dict(d=12), -2), (dict(d=264), -2),
            (dict(io_dtype=2), -3), (dict(n_nodes=1024, h_q=200), -2)]
BAD_CACHE = [(dict(k=None), -1), (dict(v=None), -1), (dict(k=ODD), -5), (dict(io_dtype=7), -3), (dict(io_dtype=1), -3),
             (dict(n_pages=0), -2), (dict(page_rows=0), -2), (dict(page_rows=65537), -2), (dict(n_layers=0), -2),
             (dict(h_kv=1), -2), (dict(d=40), -2), (dict(k_row=66), -5), (dict(v_head=33), -5), (dict(v_page=-1024), -2)]


@NO_GPU
def test_verify_refusals():
    def call(d=dims(), off=None, c=cache(), layer=0, table=FAKE, width=4, ctx=FAKE, q=rows(), k=rows(), v=rows(),
             anc=FAKE, status=FAKE, o=rows(), ws=FAKE):
        r = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
        return T._lib.gdn_attn_verify(r(d), off, r(c), layer, table, width, ctx, r(q), r(k), r(v), anc, status, r(o),
                                      ws, None)
    assert call(d=None) == -1
    for kw, rc in BAD_DIMS + [(dict(scale=0.0), -2), (dict(scale=-1.0), -2), (dict(scale=float("nan")), -2),
                              (dict(scale=float("inf")), -2)]:
        assert call(d=dims(**kw)) == rc, kw
    for kw, rc in BAD_CACHE:
        assert call(c=cache(**kw)) == rc, kw
    assert call(c=None) == -1
    for name in ("table", "ctx", "anc", "status", "ws"):
        assert call(**{name: None}) == -1 and call(**{name: ODD}) == -5, name
    for name in ("q", "k", "v", "o"):
        assert call(**{name: None}) == -1 and call(**{name: rows(None)}) == -1, name
        assert call(**{name: rows(ODD)}) == -5 and call(**{name: rows(row=66)}) == -5, name
        assert call(**{name: rows(head=-32)}) == -2, name
    assert call(layer=1) == -2 and call(layer=-1) == -2 and call(width=-1) == -2
    assert call(off=FAKE + 2) == -5
    assert call(d=dims(batch=0), c=None, q=None) == 0


@NO_GPU
def test_rope_refusals():
    def call(d=dims(), rp=T.RopeDims(32, 0, 1.0), off=None, n=6, q=rows(), k=rows(), freq=FAKE, ctx=FAKE, depth=FAKE,
             qo=rows(), ko=rows()):
        r = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
        return T._lib.gdn_attn_rope(r(d), r(rp), off, n, r(q), r(k), freq, ctx, depth, r(qo), r(ko), None)
    assert call(d=None) == -1 and call(rp=None) == -1
    for kw, rc in BAD_DIMS:
        assert call(d=dims(**kw)) == rc, kw
    for rot, layout, amp in ((0, 0, 1.0), (3, 0, 1.0), (34, 0, 1.0), (32, 2, 1.0), (32, 0, float("nan"))):
        assert call(rp=T.RopeDims(rot, layout, amp)) == -2
    for name in ("q", "k", "qo", "ko"):
        assert call(**{name: None}) == -1 and call(**{name: rows(ODD)}) == -5 and call(**{name: rows(row=2)}) == -5
    for name in ("freq", "ctx", "depth"):
        assert call(**{name: None}) == -1 and call(**{name: ODD}) == -5
    assert call(n=-1) == -2 and call(n=2 ** 31) == -2 and call(n=0) == 0 and call(off=FAKE + 1) == -5


@NO_GPU
def test_commit_refusals():
    def call(d=dims(), off=None, c=cache(), layer=0, table=FAKE, width=4, ctx=FAKE, k=rows(), v=rows(), path=FAKE,
             path_len=FAKE, new_len=FAKE + 64):
        r = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
        return T._lib.gdn_attn_commit(r(d), off, r(c), layer, table, width, ctx, r(k), r(v), path, path_len, new_len,
                                      None)
    for kw, rc in BAD_DIMS:
        assert call(d=dims(**kw)) == rc, kw
    for kw, rc in BAD_CACHE:
        assert call(c=cache(**kw)) == rc, kw
    for name in ("table", "ctx", "path", "path_len", "new_len"):
        assert call(**{name: None}) == -1 and call(**{name: ODD}) == -5, name
    assert call(new_len=FAKE) == -6


@NO_GPU
def test_pages_refusals():
    good = T.page_dims(10, 16, 4, 3)
    L = T._lib
    calls = {"gdn_pages_fork": ((2,), 7), "gdn_pages_reserve": ((), 9), "gdn_pages_free": ((), 5),
             "gdn_pages_compact": ((4,), 7)}
    for name, (lead, n) in calls.items():
        f = lambda d, p, lead=lead, name=name: getattr(L, name)(  # noqa: E731
            ctypes.byref(d) if d else None, *lead, *p, None)
        assert f(None, [FAKE] * n) == -1
        for bad in ((0, 16, 4, 3), (10, 0, 4, 3), (10, 16, 0, 3), (10, 16, 4097, 3), (10, 16, 4, 0),
                    (2 ** 30 + 1, 16, 4, 3), (10, 65537, 4, 3), (10, 16, 4, 2 ** 20 + 1)):
            assert f(T.page_dims(*bad), [FAKE] * n) == -2, (name, bad)
        for i in range(n):
            assert f(good, [FAKE] * i + [None] + [FAKE] * (n - i - 1)) == -1, (name, i)
            assert f(good, [FAKE] * i + [ODD] + [FAKE] * (n - i - 1)) == -5, (name, i)
    assert L.gdn_pages_fork(ctypes.byref(good), -1, *[FAKE] * 7, None) == -2
    assert L.gdn_pages_fork(ctypes.byref(good), 0, *[None] * 7, None) == 0
    assert L.gdn_pages_compact(ctypes.byref(good), 0, *[FAKE] * 7, None) == -2
    c = lambda kw, p=(FAKE,) * 3, n=2: L.gdn_pages_copy(ctypes.byref(cache(**kw)), n, *p, None)  # noqa: E731
    assert L.gdn_pages_copy(None, 2, FAKE, FAKE, FAKE, None) == -1
    assert c({}, n=-1) == -2 and c({}, n=0) == 0 and c({}, (None, FAKE, FAKE)) == -1 and c({}, (FAKE, ODD, FAKE)) == -5
    assert c(dict(d=12)) == -2 and c(dict(k_head=2)) == -5


def test_workspace_bytes():
    one = T.gdn_attn_workspace_bytes(T.attn_dims(1, 1, 8, 1, 128, "bf16"))
    many = T.gdn_attn_workspace_bytes(T.attn_dims(64, 128, 32, 4, 128, "bf16"))
    assert 0 < one < many < 1 << 28
    assert T.gdn_attn_workspace_bytes(T.attn_dims(0, 1, 8, 1, 128, "bf16")) == 0
    with pytest.raises(T.GdnError):
        T.gdn_attn_workspace_bytes(T.attn_dims(1, 1, 8, 3, 128, "bf16"))


def test_binding_refuses_host_tensors():
    d = T.attn_dims(1, 2, 2, 1, 64, "f32")
    x = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError):
        T.PagedCache(torch.zeros(2, 16, 1, 64), torch.zeros(2, 16, 1, 64))
    with pytest.raises(ValueError):
        T.gdn_attn_rope(d, T.rope_dims(64), x, x[:, :1], torch.zeros(32, dtype=torch.float64),
                        torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32), x, x[:, :1])


def test_reference_attention_is_softmax():
    """The tests' reference against another formulation, and its masks."""
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 2, 8)), rng.standard_normal((7, 8)), rng.standard_normal((7, 8))
    par = parents(rng, "rrt", 3)
    look = np.concatenate([np.ones((3, 4), dtype=bool), ancestors(par) | np.eye(3, dtype=bool)], axis=1)
    o, tol = attend(q, k, v, look, 0.3, "f32")
    t = torch.softmax(torch.from_numpy(np.where(look[:, None], q @ k.T * 0.3, -np.inf)), -1).numpy() @ v
    assert np.abs(o - t).max() < 1e-12 and (tol > 0).all() and tol.max() < 1e-4
    bits = pack_bits(ancestors(par), 40)
    assert bits.shape == (40, 2) and not bits[3:].any() and not bits[:, 1].any()


def test_reference_bookkeeping_keeps_the_pool_whole():
    """Fork, reserve and free leave every page counted as often as it is held."""
    rng = np.random.default_rng(1)
    ref, table = [0] * 40, [[-1] * 6 for _ in range(9)]
    held, length = [0] * 9, [0] * 9
    for step in range(200):
        R.reserve(4, 6, rng.integers(0, 5, size=9).tolist(), ref, table, held, length)
        for s in range(9):
            length[s] = min(held[s] * 4, length[s] + int(rng.integers(0, 4)))
        R.free((rng.random(9) < 0.3).astype(int).tolist(), ref, table, held, length)
        R.fork(4, 6, rng.integers(0, 9, size=3).tolist(), rng.integers(0, 9, size=3).tolist(), ref, table, held, length)
        if step % 5 == 0:
            R.compact(100, ref, table)
        flat = [p for s in range(9) for p in table[s][:held[s]]]
        assert ref == [flat.count(p) for p in range(40)]
