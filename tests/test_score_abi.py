"""The score calls' symbols, struct layout and host-side refusals.  CPU only: no call here reaches a kernel
launch."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_score.h")

T = pytest.importorskip("tree_masked_gated_amd")
NO_GPU = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                            reason="fake device pointers are only passed where no GPU exists")
FAKE, ODD = 0x10000, 0x10004
NULL, DIMS, DTYPE, ALIGN = -1, -2, -3, -5
ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731


def test_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\bint (gdn_\w+)\s*\(", src)))
    assert names == ["gdn_score_workspace_bytes", "gdn_token_scores", "gdn_token_scores_backward"]
    out = subprocess.run(["nm", "-D", "--defined-only", T.lib_path], capture_output=True, text=True, check=True).stdout
    assert set(names) <= set(re.findall(r"\sT\s(\w+)", out))
    assert all(n in T.__all__ for n in names)


def test_header_compiles_as_c_and_struct_matches():
    lines = ["#include <stddef.h>", '#include "gdn_score.h"',
             f"_Static_assert(sizeof(gdn_score_dims) == {ctypes.sizeof(T.ScoreDims)}, \"size\");"]
    lines += [f"_Static_assert(offsetof(gdn_score_dims, {f}) == {getattr(T.ScoreDims, f).offset}, \"{f}\");"
              for f, _ in T.ScoreDims._fields_]
    p = subprocess.run(["gcc", "-x", "c", "-std=c11", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), "-I",
                        "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-"], input="\n".join(lines) + "\n", text=True,
                       capture_output=True)
    assert p.returncode == 0, p.stderr


def dims(**kw):
    return T.ScoreDims(**{**dict(rows=4, row_stride=100, vocab=100, topk=3, io_dtype=0), **kw})


BAD = [(dict(rows=-1), DIMS), (dict(rows=2 ** 22 + 1), DIMS), (dict(vocab=0), DIMS), (dict(row_stride=99), DIMS),
       (dict(vocab=2 ** 24 + 1, row_stride=2 ** 25), DIMS), (dict(topk=-1), DIMS), (dict(topk=65), DIMS),
       (dict(vocab=2, topk=3), DIMS), (dict(io_dtype=2), DTYPE), (dict(row_stride=2 ** 41), DIMS),
       (dict(rows=2 ** 22, vocab=2 ** 17, row_stride=2 ** 17), DIMS)]


@NO_GPU
def test_scores_refusals():
    def call(d=dims(), x=FAKE, tokens=FAKE, logp=FAKE, entropy=FAKE, lse=FAKE, top_logp=FAKE, top_tok=FAKE, ws=FAKE):
        return T._lib.gdn_token_scores(ref(d), x, tokens, logp, entropy, lse, top_logp, top_tok, ws, None)
    assert call(d=None) == NULL and call(x=None) == NULL and call(logp=None) == NULL
    assert call(top_logp=None) == NULL and call(top_tok=None) == NULL
    for kw, rc in BAD:
        assert call(d=dims(**kw)) == rc, kw
    for name in ("x", "tokens", "logp", "entropy", "lse", "top_logp", "top_tok", "ws"):
        assert call(**{name: ODD}) == ALIGN, name
    assert call(d=dims(rows=1, vocab=50000, row_stride=50000), ws=None) == NULL     # a row in parts needs one
    assert call(d=dims(rows=0), x=None) == 0


@NO_GPU
def test_gradient_refusals():
    def call(d=dims(), x=FAKE, tokens=FAKE, lse=FAKE, entropy=FAKE, d_logp=FAKE, d_entropy=FAKE, top_tok=FAKE,
             d_top=FAKE, out=FAKE):
        return T._lib.gdn_token_scores_backward(ref(d), x, tokens, lse, entropy, d_logp, d_entropy, top_tok, d_top, out,
                                                None)
    assert call(d=None) == NULL
    for kw, rc in BAD:
        assert call(d=dims(**kw)) == rc, kw
    # tokens with their gradient, entropy with its, alternatives with theirs
    for name in ("x", "lse", "out", "tokens", "d_logp", "entropy", "top_tok", "d_top"):
        assert call(**{name: None}) == NULL, name
    for name in ("x", "tokens", "lse", "entropy", "d_logp", "d_entropy", "top_tok", "d_top", "out"):
        assert call(**{name: ODD}) == ALIGN, name
    assert call(d=dims(rows=0), x=None) == 0


def test_workspace_sizes():
    assert T.gdn_score_workspace_bytes(T.score_dims(5000, 1000, 8, "bf16")) == 0
    assert T.gdn_score_workspace_bytes(T.score_dims(1, 150000, 8, "bf16")) > 0
    out = ctypes.c_size_t()
    assert T._lib.gdn_score_workspace_bytes(None, ctypes.byref(out)) == NULL
    assert T._lib.gdn_score_workspace_bytes(ctypes.byref(dims()), None) == NULL
    for kw, rc in BAD:
        assert T._lib.gdn_score_workspace_bytes(ctypes.byref(dims(**kw)), ctypes.byref(out)) == rc, kw


def test_binding_checks():
    d = T.score_dims(2, 10, 0, "f32")
    v, ws = torch.zeros(2), torch.empty(16, dtype=torch.uint8)
    for x in (torch.zeros(2, 10), torch.zeros(2, 11), torch.zeros(2, 10).half()):
        with pytest.raises(ValueError):
            T.gdn_token_scores(d, x, None, None, v, v, ws)
