"""The rule calls' symbols, struct layouts, sizes and host-side refusals.  CPU only: no call here reaches a
kernel launch."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_rule.h")

T = pytest.importorskip("tree_masked_gated_amd")
NO_GPU = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                            reason="fake device pointers are only passed where no GPU exists")
FAKE = 0x10000
NULL, DIMS, DTYPE, ALIGN, ALIAS = -1, -2, -3, -5, -6


def test_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\bint (gdn_\w+)\s*\(", src)))
    assert names == ["gdn_rule_backward", "gdn_rule_forward", "gdn_rule_step", "gdn_rule_workspace_bytes"]
    out = subprocess.run(["nm", "-D", "--defined-only", T.lib_path], capture_output=True, text=True, check=True).stdout
    assert set(names) <= set(re.findall(r"\sT\s(\w+)", out))
    assert all(n in T.__all__ for n in names)


def test_header_compiles_as_c_and_struct_matches():
    lines = ["#include <stddef.h>", '#include "gdn_rule.h"',
             f"_Static_assert(sizeof(gdn_rule_dims) == {ctypes.sizeof(T.RuleDims)}, \"size\");"]
    lines += [f"_Static_assert(offsetof(gdn_rule_dims, {f}) == {getattr(T.RuleDims, f).offset}, \"{f}\");"
              for f, _ in T.RuleDims._fields_]
    p = subprocess.run(["gcc", "-x", "c", "-std=c11", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), "-I",
                        "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-"], input="\n".join(lines) + "\n", text=True,
                       capture_output=True)
    assert p.returncode == 0, p.stderr


def dims(**kw):
    return T.RuleDims(**{**dict(batch=2, h_k=2, h_v=4, d_k=32, d_v=32, io_dtype=0), **kw})


def at(i):
    return FAKE + 4096 * i


def rows(data, row=128, head=32):
    return None if data is None else T.AttnRows(data, row, head)


BAD_DIMS = [(dict(batch=-1), DIMS), (dict(batch=2 ** 20 + 1), DIMS), (dict(h_k=0), DIMS), (dict(h_v=3), DIMS),
            (dict(h_k=1, h_v=2 ** 15 + 1), DIMS), (dict(d_k=0), DIMS), (dict(d_k=257), DIMS), (dict(d_v=257), DIMS),
            (dict(d_v=0), DIMS), (dict(io_dtype=2), DTYPE)]
ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731


def forward(d=dims(), off=FAKE, n=6, S0=at(1), q=rows(at(2)), k=rows(at(3)), v=rows(at(4)), beta=at(5), g=at(6),
            o=rows(at(7)), S_out=at(8), ws=at(9)):
    return T._lib.gdn_rule_forward(ref(d), off, n, S0, ref(q), ref(k), ref(v), beta, g, ref(o), S_out, ws, None)


def backward(d=dims(), off=FAKE, n=6, S0=at(1), q=rows(at(2)), k=rows(at(3)), v=rows(at(4)), beta=at(5), g=at(6),
             d_o=rows(at(7)), dS_out=at(8), dq=rows(at(9)), dk=rows(at(10)), dv=rows(at(11)), dbeta=at(12),
             dlog_g=at(13), dS0=at(14), ws=at(15)):
    return T._lib.gdn_rule_backward(ref(d), off, n, S0, ref(q), ref(k), ref(v), beta, g, ref(d_o), dS_out, ref(dq),
                                    ref(dk), ref(dv), dbeta, dlog_g, dS0, ws, None)


def step(d=dims(), slot=FAKE, n=4, q=rows(at(2)), k=rows(at(3)), v=rows(at(4)), beta=at(5), g=at(6), state=at(7),
         o=rows(at(8))):
    return T._lib.gdn_rule_step(ref(d), slot, n, ref(q), ref(k), ref(v), beta, g, state, ref(o), None)


@NO_GPU
@pytest.mark.parametrize("call,names,may,tensors", [
    (forward, ("beta", "g", "ws"), ("S0", "S_out"), ("q", "k", "v", "o")),
    (backward, ("beta", "g", "ws", "dbeta", "dlog_g"), ("S0", "dS_out", "dS0"),
     ("q", "k", "v", "d_o", "dq", "dk", "dv")),
    (step, ("beta", "g", "state"), (), ("q", "k", "v", "o"))])
def test_refusals(call, names, may, tensors):
    assert call(d=None) == NULL
    for kw, rc in BAD_DIMS:
        assert call(d=dims(**kw)) == rc, kw
    for name in names:
        assert call(**{name: None}) == NULL and call(**{name: FAKE + 4}) == ALIGN, name
    for name in may:
        assert call(**{name: FAKE + 4}) == ALIGN, name
    for name in tensors:
        assert call(**{name: None}) == NULL and call(**{name: rows(0)}) == NULL, name
        assert call(**{name: rows(FAKE + 2)}) == ALIGN, name
        assert call(**{name: rows(FAKE, row=-1)}) == DIMS and call(**{name: rows(FAKE, head=-1)}) == DIMS, name
    assert call(d=dims(batch=0), q=None, g=None) == 0


@NO_GPU
def test_refusals_of_sequences():
    for call in (forward, backward):
        assert call(off=None) == NULL and call(off=FAKE + 2) == ALIGN
        assert call(n=-1) == DIMS and call(n=2 ** 31) == DIMS and call(n=2 ** 27 + 64) == DIMS
        assert call(d=dims(batch=2 ** 20, h_k=16, h_v=16)) == DIMS
    # an output that is an input, or another output
    assert forward(o=rows(at(2))) == ALIAS and forward(S_out=at(4)) == ALIAS and forward(o=rows(at(1))) == ALIAS
    for name, other in (("dq", 2), ("dk", 9), ("dv", 7), ("dq", 8), ("dk", 1)):
        assert backward(**{name: rows(at(other))}) == ALIAS, name
    for name, other in (("dbeta", 5), ("dlog_g", 12), ("dS0", 1), ("dS0", 13)):
        assert backward(**{name: at(other)}) == ALIAS, name


@NO_GPU
def test_refusals_of_a_step():
    assert step(slot=FAKE + 2) == ALIGN
    assert step(n=-1) == DIMS and step(slot=None, n=1) == DIMS
    assert step(d=dims(batch=65536)) == DIMS
    assert step(o=rows(at(2))) == ALIAS and step(state=at(5)) == ALIAS and step(o=rows(at(7))) == ALIAS


def test_workspace_sizes():
    d = T.rule_dims(3, 2, 4, 100, 33, "bf16")
    small, large, back = (T.gdn_rule_workspace_bytes(d, *x) for x in ((0,), (1000,), (1000, True)))
    assert 0 < small < large < back
    assert T.gdn_rule_workspace_bytes(d, 999) <= large          # never more for fewer rows
    out = ctypes.c_size_t()
    assert T._lib.gdn_rule_workspace_bytes(None, 1, 0, ctypes.byref(out)) == NULL
    assert T._lib.gdn_rule_workspace_bytes(ctypes.byref(d), 1, 0, None) == NULL
    assert T._lib.gdn_rule_workspace_bytes(ctypes.byref(d), -1, 0, ctypes.byref(out)) == DIMS
    for kw, rc in BAD_DIMS:
        assert T._lib.gdn_rule_workspace_bytes(ctypes.byref(dims(**kw)), 1, 0, ctypes.byref(out)) == rc


@pytest.mark.parametrize("bad", ["shape", "dtype", "host", "strided"])
def test_binding_checks(bad):
    """The binding refuses what the C call could not see.  Host tensors everywhere: the first check to fail is
    the device's, except for what is checked before it."""
    d = T.rule_dims(1, 1, 1, 8, 8, "f32")
    x = torch.zeros(4, 1, 8)
    if bad == "shape":
        x = torch.zeros(4, 2, 8)
    elif bad == "dtype":
        x = x.half()
    elif bad == "strided":
        x = torch.zeros(4, 1, 16)[..., ::2]
    gate, off = torch.zeros(4, 1), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises((ValueError, TypeError)):
        T.gdn_rule_forward(d, off, x, x, x, gate, gate, x.clone(), torch.empty(16, dtype=torch.uint8))
