"""Python binding of libgdntree.so: rollback-free GDN draft-tree verification on
MI355X (gfx950).

The names mirror the C ABI in include/gdn_tree.h and include/gdn_attn.h.  This module only marshals
arguments: it checks that each torch tensor has the shape, dtype and
contiguity the C ABI documents (so a kernel never reads past a buffer) and
passes device pointers and the current HIP stream.  Every step of the
computation runs in the library's HIP kernels; there is no other path.  PyTorch
provides device memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Dict, Optional

__all__ = [
    "GDN_F32", "GDN_BF16", "GdnError", "Dims", "Cache", "lib_path", "dims",
    "gdn_tree_cache_bytes", "gdn_tree_verify", "gdn_tree_commit", "gdn_tree_commit_verify",
    "gdn_tree_accept", "gdn_tree_verify_ragged", "gdn_tree_commit_ragged",
    "gdn_tree_commit_verify_ragged", "gdn_tree_accept_ragged", "check_offsets",
    "BuildDims", "build_dims", "gdn_tree_build",
    "gdn_tree_strerror", "TreeCache",
    "ROPE_HALF", "ROPE_INTERLEAVED", "AttnDims", "RopeDims", "PageDims", "AttnRows", "PagedCacheStruct",
    "PagedCache", "attn_dims", "rope_dims", "page_dims", "attn_workspace", "gdn_attn_workspace_bytes",
    "gdn_attn_rope", "gdn_attn_verify", "gdn_attn_commit", "gdn_pages_fork", "gdn_pages_reserve",
    "gdn_pages_copy", "gdn_pages_free", "gdn_pages_compact",
]

GDN_F32, GDN_BF16 = 0, 1
_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libgdntree.so")

if not os.path.exists(lib_path):
    raise ImportError(
        f"{lib_path} is missing: build the HIP library first "
        "(python tree_masked_gated_amd/build.py)")


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "n_nodes", "h_k", "h_v", "d_k", "d_v", "io_dtype")]


class BuildDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "n_nodes", "topk", "width")]


class Cache(ctypes.Structure):
    _fields_ = [("anc_mask", ctypes.c_void_p), ("depth", ctypes.c_void_p),
                ("u", ctypes.c_void_p), ("log_gamma", ctypes.c_void_p),
                ("tree_status", ctypes.c_void_p)]


# torch first: its bundled HIP runtime (soname libamdhip64.so.7) then also
# serves this library, so tensors and kernels share one runtime.  Loading the
# library first would pull in a second runtime that cannot see torch's memory.
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(lib_path)
_vp, _i = ctypes.c_void_p, ctypes.c_int
_sz = ctypes.POINTER(ctypes.c_size_t)
_lib.gdn_tree_cache_bytes.argtypes = [ctypes.POINTER(Dims), _sz, _sz, _sz, _sz, _sz]
_lib.gdn_tree_cache_bytes.restype = _i
_lib.gdn_tree_verify.argtypes = [ctypes.POINTER(Dims)] + [_vp] * 8 + [ctypes.POINTER(Cache), _vp]
_lib.gdn_tree_verify.restype = _i
_lib.gdn_tree_commit.argtypes = [ctypes.POINTER(Dims)] + [_vp] * 3 + \
    [ctypes.POINTER(Cache)] + [_vp] * 3 + [_vp]
_lib.gdn_tree_commit.restype = _i
_lib.gdn_tree_commit_verify.argtypes = [ctypes.POINTER(Dims)] + [_vp] * 3 + [ctypes.POINTER(Cache)] + \
    [_vp] * 10 + [ctypes.POINTER(Cache), _vp]
_lib.gdn_tree_commit_verify.restype = _i
_lib.gdn_tree_accept.argtypes = [ctypes.POINTER(Dims)] + [_vp] * 7 + [_vp]
_lib.gdn_tree_accept.restype = _i
_lib.gdn_tree_verify_ragged.argtypes = [ctypes.POINTER(Dims)] + [_vp] * 9 + [ctypes.POINTER(Cache), _vp]
_lib.gdn_tree_verify_ragged.restype = _i
_lib.gdn_tree_commit_ragged.argtypes = [ctypes.POINTER(Dims)] + [_vp] * 4 + \
    [ctypes.POINTER(Cache)] + [_vp] * 3 + [_vp]
_lib.gdn_tree_commit_ragged.restype = _i
_lib.gdn_tree_commit_verify_ragged.argtypes = [ctypes.POINTER(Dims)] + [_vp] * 4 + \
    [ctypes.POINTER(Cache)] + [_vp] * 11 + [ctypes.POINTER(Cache), _vp]
_lib.gdn_tree_commit_verify_ragged.restype = _i
_lib.gdn_tree_accept_ragged.argtypes = [ctypes.POINTER(Dims)] + [_vp] * 8 + [_vp]
_lib.gdn_tree_accept_ragged.restype = _i
_lib.gdn_tree_build.argtypes = [ctypes.POINTER(BuildDims)] + [_vp] * 5 + [_vp]
_lib.gdn_tree_build.restype = _i
_lib.gdn_tree_strerror.argtypes = [_i]
_lib.gdn_tree_strerror.restype = ctypes.c_char_p


class GdnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {gdn_tree_strerror(code)} ({code})")
        self.code = code


def gdn_tree_strerror(code: int) -> str:
    return _lib.gdn_tree_strerror(int(code)).decode()


def dims(batch, n_nodes, h_k, h_v, d_k, d_v, io_dtype) -> Dims:
    if isinstance(io_dtype, str):
        io_dtype = {"f32": GDN_F32, "bf16": GDN_BF16}[io_dtype]
    return Dims(batch, n_nodes, h_k, h_v, d_k, d_v, io_dtype)


def gdn_tree_cache_bytes(d: Dims) -> Dict[str, int]:
    out = [ctypes.c_size_t() for _ in range(5)]
    rc = _lib.gdn_tree_cache_bytes(ctypes.byref(d), *[ctypes.byref(x) for x in out])
    if rc:
        raise GdnError(rc, "gdn_tree_cache_bytes")
    return dict(zip(("anc_mask", "depth", "u", "log_gamma", "tree_status"),
                    (x.value for x in out)))


# ------------------------------------------------------------ marshalling

_int32 = torch.int32


def _torch():
    return torch


def _io_dtype(d: Dims):
    torch = _torch()
    return torch.float32 if d.io_dtype == GDN_F32 else torch.bfloat16


def _ptr(x, shape, dtype, name):
    """Device pointer of x after checking it covers the documented layout.
    Raw integers are taken as device pointers as they are; None gives NULL."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor or a device pointer")
    if not x.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if x.dtype != dtype:
        raise ValueError(f"{name}: dtype {x.dtype}, expected {dtype}")
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return x.data_ptr()


# The current stream's handle without its stream object, which takes 3 us of an 11 us call.  The function is
# torch's own and not part of its public interface: where it is gone, the object is made.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class TreeCache:
    """Device buffers of a gdn_tree_cache for one Dims, allocated with torch
    (allocation is plumbing; the library itself allocates nothing)."""

    def __init__(self, d: Dims, device="cuda"):
        torch = _torch()
        B, N, Hv, dv = d.batch, d.n_nodes, d.h_v, d.d_v
        W = (N + 31) // 32
        self.dims = d
        self.anc_mask = torch.zeros((B, N, W), dtype=torch.int32, device=device)
        self.depth = torch.zeros((B, N), dtype=torch.int32, device=device)
        self.u = torch.zeros((B, Hv, N, dv), dtype=torch.float32, device=device)
        self.log_gamma = torch.zeros((B, Hv, N), dtype=torch.float32, device=device)
        self.tree_status = torch.zeros((B,), dtype=torch.int32, device=device)
        sizes = gdn_tree_cache_bytes(d)
        for key, size in sizes.items():
            t = getattr(self, key)
            assert t.numel() * t.element_size() == size, key
        self.struct = Cache(*(getattr(self, key).data_ptr() for key in
                              ("anc_mask", "depth", "u", "log_gamma", "tree_status")))


def _cache_struct(cache):
    if isinstance(cache, TreeCache):
        return cache.struct
    if isinstance(cache, Cache):
        return cache
    raise TypeError("cache: expected TreeCache or Cache")


def gdn_tree_verify(d: Dims, S0, q, k, v, beta, g, parent, o, cache, stream=None) -> None:
    """Enqueue verification of every node of every tree (see gdn_tree.h)."""
    torch = _torch()
    B, N, Hk, Hv, dk, dv = d.batch, d.n_nodes, d.h_k, d.h_v, d.d_k, d.d_v
    io = _io_dtype(d)
    if isinstance(cache, TreeCache):
        _check_cache(cache, d)
    args = [
        _ptr(S0, (B, Hv, dv, dk), torch.float32, "S0"),
        _ptr(q, (B, N, Hk, dk), io, "q"),
        _ptr(k, (B, N, Hk, dk), io, "k"),
        _ptr(v, (B, N, Hv, dv), io, "v"),
        _ptr(beta, (B, N, Hv), torch.float32, "beta"),
        _ptr(g, (B, N, Hv), torch.float32, "g"),
        _ptr(parent, (B, N), torch.int32, "parent"),
        _ptr(o, (B, N, Hv, dv), io, "o"),
    ]
    rc = _lib.gdn_tree_verify(ctypes.byref(d), *args, ctypes.byref(_cache_struct(cache)),
                              _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_tree_verify")


def gdn_tree_commit(d: Dims, S_in, S_out, k, cache, accepted, path, path_len,
                    stream=None) -> None:
    """Enqueue the commit of each sequence's accepted node (see gdn_tree.h)."""
    torch = _torch()
    B, N, Hk, Hv, dk, dv = d.batch, d.n_nodes, d.h_k, d.h_v, d.d_k, d.d_v
    if isinstance(cache, TreeCache):
        _check_cache(cache, d)
    args = [
        _ptr(S_in, (B, Hv, dv, dk), torch.float32, "S_in"),
        _ptr(S_out, (B, Hv, dv, dk), torch.float32, "S_out"),
        _ptr(k, (B, N, Hk, dk), _io_dtype(d), "k"),
    ]
    tail = [
        _ptr(accepted, (B,), torch.int32, "accepted"),
        _ptr(path, (B, N), torch.int32, "path"),
        _ptr(path_len, (B,), torch.int32, "path_len"),
    ]
    rc = _lib.gdn_tree_commit(ctypes.byref(d), *args, ctypes.byref(_cache_struct(cache)),
                              *tail, _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_tree_commit")


def gdn_tree_commit_verify(d: Dims, S_prev, S_new, k_prev, cache_prev, accepted_prev, path_prev,
                           path_len_prev, q, k, v, beta, g, parent, o, cache, stream=None) -> None:
    """Enqueue the previous tree's commit and the new tree's verification as one
    step, the committed state used directly as the new prefix state (see
    gdn_tree.h)."""
    torch = _torch()
    B, N, Hk, Hv, dk, dv = d.batch, d.n_nodes, d.h_k, d.h_v, d.d_k, d.d_v
    io = _io_dtype(d)
    for c in (cache_prev, cache):
        if isinstance(c, TreeCache):
            _check_cache(c, d)
    head = [
        _ptr(S_prev, (B, Hv, dv, dk), torch.float32, "S_prev"),
        _ptr(S_new, (B, Hv, dv, dk), torch.float32, "S_new"),
        _ptr(k_prev, (B, N, Hk, dk), io, "k_prev"),
    ]
    mid = [
        _ptr(accepted_prev, (B,), torch.int32, "accepted_prev"),
        _ptr(path_prev, (B, N), torch.int32, "path_prev"),
        _ptr(path_len_prev, (B,), torch.int32, "path_len_prev"),
        _ptr(q, (B, N, Hk, dk), io, "q"),
        _ptr(k, (B, N, Hk, dk), io, "k"),
        _ptr(v, (B, N, Hv, dv), io, "v"),
        _ptr(beta, (B, N, Hv), torch.float32, "beta"),
        _ptr(g, (B, N, Hv), torch.float32, "g"),
        _ptr(parent, (B, N), torch.int32, "parent"),
        _ptr(o, (B, N, Hv, dv), io, "o"),
    ]
    rc = _lib.gdn_tree_commit_verify(ctypes.byref(d), *head, ctypes.byref(_cache_struct(cache_prev)),
                                     *mid, ctypes.byref(_cache_struct(cache)), _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_tree_commit_verify")


def gdn_tree_accept(d: Dims, parent, draft, target, target_root, accepted, accept_len, next_token,
                    stream=None) -> None:
    """Enqueue the greedy acceptance walk (see gdn_tree.h)."""
    torch = _torch()
    B, N = d.batch, d.n_nodes
    ptrs = [
        _ptr(parent, (B, N), torch.int32, "parent"),
        _ptr(draft, (B, N), torch.int32, "draft"),
        _ptr(target, (B, N), torch.int32, "target"),
        _ptr(target_root, (B,), torch.int32, "target_root"),
        _ptr(accepted, (B,), torch.int32, "accepted"),
        _ptr(accept_len, (B,), torch.int32, "accept_len"),
        _ptr(next_token, (B,), torch.int32, "next_token"),
    ]
    rc = _lib.gdn_tree_accept(ctypes.byref(d), *ptrs, _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_tree_accept")


# ---------------------------------------------------------------- ragged batches
# Per-node arrays packed sequence after sequence: T rows in all (the leading
# extent of every per-node tensor, taken from the first one), sequence b owning
# rows offsets[b] .. offsets[b+1] - 1 (offsets: int32 [B + 1] on the device).


def check_offsets(offsets, d: Dims, T: int) -> None:
    """Host-side check (copies offsets to the host and so synchronises) that
    the offsets describe B trees of at most N nodes inside T rows.  The library
    itself only checks each sequence's own count on the device; an offsets
    array that points past T rows is the caller's error."""
    o = offsets.cpu().tolist() if hasattr(offsets, "cpu") else list(offsets)
    if len(o) != d.batch + 1 or o[0] != 0:
        raise ValueError("offsets: expected B + 1 entries starting at 0")
    if any(b < a or b - a > d.n_nodes for a, b in zip(o, o[1:])):
        raise ValueError("offsets: non-decreasing, at most n_nodes rows per sequence")
    if o[-1] > T:
        raise ValueError(f"offsets: {o[-1]} rows, arrays hold {T}")


def _rows(x, name):
    if isinstance(x, int) or x is None:
        raise TypeError(f"{name}: ragged calls take tensors (their leading extent is T)")
    return int(x.shape[0])


def gdn_tree_verify_ragged(d: Dims, offsets, S0, q, k, v, beta, g, parent, o, cache,
                           stream=None) -> None:
    """Enqueue verification of a batch of trees of different sizes (see
    gdn_tree.h, ragged batches)."""
    torch = _torch()
    B, Hk, Hv, dk, dv = d.batch, d.h_k, d.h_v, d.d_k, d.d_v
    T = _rows(q, "q")
    io = _io_dtype(d)
    if isinstance(cache, TreeCache):
        _check_cache(cache, d)
    args = [
        _ptr(offsets, (B + 1,), torch.int32, "offsets"),
        _ptr(S0, (B, Hv, dv, dk), torch.float32, "S0"),
        _ptr(q, (T, Hk, dk), io, "q"),
        _ptr(k, (T, Hk, dk), io, "k"),
        _ptr(v, (T, Hv, dv), io, "v"),
        _ptr(beta, (T, Hv), torch.float32, "beta"),
        _ptr(g, (T, Hv), torch.float32, "g"),
        _ptr(parent, (T,), torch.int32, "parent"),
        _ptr(o, (T, Hv, dv), io, "o"),
    ]
    rc = _lib.gdn_tree_verify_ragged(ctypes.byref(d), *args, ctypes.byref(_cache_struct(cache)),
                                     _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_tree_verify_ragged")


def gdn_tree_commit_ragged(d: Dims, offsets, S_in, S_out, k, cache, accepted, path, path_len,
                           stream=None) -> None:
    """Enqueue the commit of each sequence's accepted node, ragged layout."""
    torch = _torch()
    B, Hk, Hv, dk, dv = d.batch, d.h_k, d.h_v, d.d_k, d.d_v
    T = _rows(k, "k")
    if isinstance(cache, TreeCache):
        _check_cache(cache, d)
    args = [
        _ptr(offsets, (B + 1,), torch.int32, "offsets"),
        _ptr(S_in, (B, Hv, dv, dk), torch.float32, "S_in"),
        _ptr(S_out, (B, Hv, dv, dk), torch.float32, "S_out"),
        _ptr(k, (T, Hk, dk), _io_dtype(d), "k"),
    ]
    tail = [
        _ptr(accepted, (B,), torch.int32, "accepted"),
        _ptr(path, (T,), torch.int32, "path"),
        _ptr(path_len, (B,), torch.int32, "path_len"),
    ]
    rc = _lib.gdn_tree_commit_ragged(ctypes.byref(d), *args, ctypes.byref(_cache_struct(cache)),
                                     *tail, _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_tree_commit_ragged")


def gdn_tree_commit_verify_ragged(d: Dims, offsets_prev, S_prev, S_new, k_prev, cache_prev,
                                  accepted_prev, path_prev, path_len_prev, offsets, q, k, v, beta,
                                  g, parent, o, cache, stream=None) -> None:
    """Enqueue the previous tree's commit and the new tree's verification as one
    step, ragged layout (each tree its own offsets)."""
    torch = _torch()
    B, Hk, Hv, dk, dv = d.batch, d.h_k, d.h_v, d.d_k, d.d_v
    Tp, T = _rows(k_prev, "k_prev"), _rows(q, "q")
    io = _io_dtype(d)
    for c in (cache_prev, cache):
        if isinstance(c, TreeCache):
            _check_cache(c, d)
    head = [
        _ptr(offsets_prev, (B + 1,), torch.int32, "offsets_prev"),
        _ptr(S_prev, (B, Hv, dv, dk), torch.float32, "S_prev"),
        _ptr(S_new, (B, Hv, dv, dk), torch.float32, "S_new"),
        _ptr(k_prev, (Tp, Hk, dk), io, "k_prev"),
    ]
    mid = [
        _ptr(accepted_prev, (B,), torch.int32, "accepted_prev"),
        _ptr(path_prev, (Tp,), torch.int32, "path_prev"),
        _ptr(path_len_prev, (B,), torch.int32, "path_len_prev"),
        _ptr(offsets, (B + 1,), torch.int32, "offsets"),
        _ptr(q, (T, Hk, dk), io, "q"),
        _ptr(k, (T, Hk, dk), io, "k"),
        _ptr(v, (T, Hv, dv), io, "v"),
        _ptr(beta, (T, Hv), torch.float32, "beta"),
        _ptr(g, (T, Hv), torch.float32, "g"),
        _ptr(parent, (T,), torch.int32, "parent"),
        _ptr(o, (T, Hv, dv), io, "o"),
    ]
    rc = _lib.gdn_tree_commit_verify_ragged(ctypes.byref(d), *head,
                                            ctypes.byref(_cache_struct(cache_prev)), *mid,
                                            ctypes.byref(_cache_struct(cache)), _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_tree_commit_verify_ragged")


def gdn_tree_accept_ragged(d: Dims, offsets, parent, draft, target, target_root, accepted,
                           accept_len, next_token, stream=None) -> None:
    """Enqueue the greedy acceptance walk, ragged layout."""
    torch = _torch()
    B = d.batch
    T = _rows(parent, "parent")
    ptrs = [
        _ptr(offsets, (B + 1,), torch.int32, "offsets"),
        _ptr(parent, (T,), torch.int32, "parent"),
        _ptr(draft, (T,), torch.int32, "draft"),
        _ptr(target, (T,), torch.int32, "target"),
        _ptr(target_root, (B,), torch.int32, "target_root"),
        _ptr(accepted, (B,), torch.int32, "accepted"),
        _ptr(accept_len, (B,), torch.int32, "accept_len"),
        _ptr(next_token, (B,), torch.int32, "next_token"),
    ]
    rc = _lib.gdn_tree_accept_ragged(ctypes.byref(d), *ptrs, _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_tree_accept_ragged")


# ---------------------------------------------------------------- tree construction

def build_dims(batch, n_nodes, topk, width) -> BuildDims:
    return BuildDims(batch, n_nodes, topk, width)


def gdn_tree_build(bd: BuildDims, logp, tok, parent, token, score, stream=None) -> None:
    """Enqueue draft-tree construction with `width` expansions per step from the
    drafter's top-k continuations (see gdn_tree.h)."""
    torch = _torch()
    B, N, K = bd.batch, bd.n_nodes, bd.topk
    ptrs = [
        _ptr(logp, (B, N + 1, K), torch.float32, "logp"),
        _ptr(tok, (B, N + 1, K), torch.int32, "tok"),
        _ptr(parent, (B, N), torch.int32, "parent"),
        _ptr(token, (B, N), torch.int32, "token"),
        _ptr(score, (B, N), torch.float32, "score"),
    ]
    rc = _lib.gdn_tree_build(ctypes.byref(bd), *ptrs, _stream(stream))
    if rc:
        raise GdnError(rc, "gdn_tree_build")


def _check_cache(c: TreeCache, d: Dims):
    cd = c.dims
    if (cd.batch, cd.n_nodes, cd.h_v, cd.d_v) != (d.batch, d.n_nodes, d.h_v, d.d_v):
        raise ValueError("cache was allocated for different dims")


# ---------------------------------------------------------------- attention layers
# Softmax attention of the same trees (include/gdn_attn.h): rotary positions, attention
# over a paged cache, append of the accepted path, page bookkeeping.  Tensors of rows
# ([T, heads, d]) may be strided slices; a ragged call takes `offsets`.

ROPE_HALF, ROPE_INTERLEAVED = 0, 1


class AttnDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "n_nodes", "h_q", "h_kv", "d", "io_dtype")] + \
        [("scale", ctypes.c_float)]


class RopeDims(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("amp", ctypes.c_double)]


class PageDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_pages", "page_rows", "n_slots", "width")]


class AttnRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class PagedCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + \
        [(n, ctypes.c_int32) for n in ("n_layers", "n_pages", "page_rows", "h_kv", "d", "io_dtype")] + \
        [(n, ctypes.c_int64) for n in ("k_layer", "k_page", "k_row", "k_head",
                                       "v_layer", "v_page", "v_row", "v_head")]


_ar, _i32, _i64 = ctypes.POINTER(AttnRows), ctypes.c_int32, ctypes.c_int64
_ad, _pd, _pc = ctypes.POINTER(AttnDims), ctypes.POINTER(PageDims), ctypes.POINTER(PagedCacheStruct)
for _name, _args in {
        "gdn_attn_rope": [_ad, ctypes.POINTER(RopeDims), _vp, _i64, _ar, _ar, _vp, _vp, _vp, _ar, _ar, _vp],
        "gdn_attn_workspace_bytes": [_ad, _sz],
        "gdn_attn_verify": [_ad, _vp, _pc, _i32, _vp, _i32, _vp, _ar, _ar, _ar, _vp, _vp, _ar, _vp, _vp],
        "gdn_attn_commit": [_ad, _vp, _pc, _i32, _vp, _i32, _vp, _ar, _ar, _vp, _vp, _vp, _vp],
        "gdn_pages_fork": [_pd, _i32] + [_vp] * 8,
        "gdn_pages_reserve": [_pd] + [_vp] * 10,
        "gdn_pages_copy": [_pc, _i32] + [_vp] * 4,
        "gdn_pages_free": [_pd] + [_vp] * 6,
        "gdn_pages_compact": [_pd, _i32] + [_vp] * 8}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _i


def attn_dims(batch, n_nodes, h_q, h_kv, d, io_dtype, scale=None) -> AttnDims:
    """scale: the factor of q.k, d ** -0.5 unless given."""
    if isinstance(io_dtype, str):
        io_dtype = {"f32": GDN_F32, "bf16": GDN_BF16}[io_dtype]
    return AttnDims(batch, n_nodes, h_q, h_kv, d, io_dtype, d ** -0.5 if scale is None else scale)


def rope_dims(rot, layout="half", amp=1.0) -> RopeDims:
    if isinstance(layout, str):
        layout = {"half": ROPE_HALF, "interleaved": ROPE_INTERLEAVED}[layout]
    return RopeDims(rot, layout, amp)


def page_dims(n_pages, page_rows, n_slots, width) -> PageDims:
    return PageDims(n_pages, page_rows, n_slots, width)


class PagedCache:
    """Key and value pools as one gdn_paged_cache: tensors [pages, page_rows, h_kv, d], or
    with a leading axis of layers, of any strides with the last axis contiguous (a pool kept
    heads first is passed as its transposed view)."""

    def __init__(self, k, v):
        torch = _torch()
        if k.shape != v.shape or k.dtype != v.dtype or k.dim() not in (4, 5):
            raise ValueError("PagedCache: k and v [layers,] pages, page_rows, h_kv, d of one shape and dtype")
        if k.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"PagedCache: dtype {k.dtype}")
        if not (k.is_cuda and v.is_cuda):
            raise ValueError("PagedCache: must be device tensors")
        if k.stride(-1) != 1 or v.stride(-1) != 1:
            raise ValueError("PagedCache: the last axis must be contiguous")
        self.k, self.v = k, v
        pages, rows, heads, d = k.shape[-4:]
        lead = lambda t: (t.stride(0) if t.dim() == 5 else 0, *t.stride()[-4:-1])  # noqa: E731
        self.struct = PagedCacheStruct(
            k.data_ptr(), v.data_ptr(), k.shape[0] if k.dim() == 5 else 1, pages, rows, heads, d,
            GDN_F32 if k.dtype == torch.float32 else GDN_BF16, *lead(k), *lead(v))


def _cache_ref(cache):
    if isinstance(cache, PagedCache):
        return ctypes.byref(cache.struct)
    if isinstance(cache, PagedCacheStruct):
        return ctypes.byref(cache)
    raise TypeError("cache: expected PagedCache or PagedCacheStruct")


def _attn_rows(x, rows, heads, d, io, name):
    """gdn_attn_rows of a [rows, heads, d] tensor with a contiguous last axis."""
    if x.dtype != io or not x.is_cuda:
        raise ValueError(f"{name}: expected a device tensor of {io}")
    if x.shape != (rows, heads, d):
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {(rows, heads, d)}")
    row, head, one = x.stride()
    if one != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return AttnRows(x.data_ptr(), row, head)


def _ints(x, shape, name):
    """Device pointer of a contiguous int32 tensor of this shape."""
    if x.dtype is not _int32 or not x.is_cuda or not x.is_contiguous() or x.shape != shape:
        raise ValueError(f"{name}: expected a contiguous int32 device tensor of shape {tuple(shape)}, "
                         f"got {x.dtype} {tuple(x.shape)}")
    return x.data_ptr()


def _attn_offsets(offsets, d, x):
    """Offsets pointer and number of rows of a dense or ragged call whose first row tensor is x."""
    if offsets is None:
        return None, d.batch * d.n_nodes
    return _ints(offsets, (d.batch + 1,), "offsets"), x.shape[0]


def _call(fn, *args):
    rc = getattr(_lib, fn)(*args)
    if rc:
        raise GdnError(rc, fn)


def gdn_attn_rope(d: AttnDims, rope: RopeDims, q, k, freq, ctx, depth, q_out, k_out, offsets=None,
                  stream=None) -> None:
    """Enqueue the rotation of the trees' queries and keys to their nodes' positions (see
    gdn_attn.h).  freq: float64 [rot / 2]; depth: [B, N], TreeCache.depth."""
    torch = _torch()
    io = _io_dtype(d)
    off, T = _attn_offsets(offsets, d, q)
    if freq.dtype != torch.float64 or freq.shape != (rope.rot // 2,) or not freq.is_cuda or not freq.is_contiguous():
        raise ValueError(f"freq: expected a contiguous float64 device tensor of {rope.rot // 2} values")
    _call("gdn_attn_rope", ctypes.byref(d), ctypes.byref(rope), off, T,
          _attn_rows(q, T, d.h_q, d.d, io, "q"), _attn_rows(k, T, d.h_kv, d.d, io, "k"), freq.data_ptr(),
          _ints(ctx, (d.batch,), "ctx"), _ints(depth, (d.batch, d.n_nodes), "depth"),
          _attn_rows(q_out, T, d.h_q, d.d, io, "q_out"), _attn_rows(k_out, T, d.h_kv, d.d, io, "k_out"),
          _stream(stream))


def gdn_attn_workspace_bytes(d: AttnDims) -> int:
    out = ctypes.c_size_t()
    _call("gdn_attn_workspace_bytes", ctypes.byref(d), ctypes.byref(out))
    return out.value


def attn_workspace(d: AttnDims, device="cuda"):
    """A zeroed workspace for gdn_attn_verify calls, one after the other, of these dims or of any that need
    no more bytes (fewer sequences, smaller trees)."""
    torch = _torch()
    return torch.zeros(max(gdn_attn_workspace_bytes(d), 16), dtype=torch.uint8, device=device)


def gdn_attn_verify(d: AttnDims, cache, table, ctx, q, k, v, anc_mask, tree_status, o, workspace,
                    offsets=None, layer=0, stream=None) -> None:
    """Enqueue the attention of every node of every tree over its sequence's pages, its
    ancestors and itself (see gdn_attn.h).  anc_mask and tree_status: TreeCache's."""
    torch = _torch()
    B, N, io = d.batch, d.n_nodes, _io_dtype(d)
    off, T = _attn_offsets(offsets, d, q)
    if table.dim() != 2:
        raise ValueError("table: expected [B, width]")
    if workspace.dtype != torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous() or \
            workspace.numel() < _workspace_bytes(d):
        raise ValueError(f"workspace: expected {_workspace_bytes(d)} contiguous bytes or more (attn_workspace)")
    args = (_ints(table, (B, table.shape[1]), "table"), table.shape[1], _ints(ctx, (B,), "ctx"),
            _attn_rows(q, T, d.h_q, d.d, io, "q"), _attn_rows(k, T, d.h_kv, d.d, io, "k"),
            _attn_rows(v, T, d.h_kv, d.d, io, "v"), _ints(anc_mask, (B, N, (N + 31) // 32), "anc_mask"),
            _ints(tree_status, (B,), "tree_status"), _attn_rows(o, T, d.h_q, d.d, io, "o"))
    if T == 0:                                   # trees without nodes: no row of o
        return
    _call("gdn_attn_verify", ctypes.byref(d), off, _cache_ref(cache), layer, *args, workspace.data_ptr(),
          _stream(stream))


@functools.lru_cache(maxsize=None)
def _workspace_bytes_of(*sizes):
    return gdn_attn_workspace_bytes(AttnDims(*sizes, 1.0))


def _workspace_bytes(d: AttnDims) -> int:
    return _workspace_bytes_of(d.batch, d.n_nodes, d.h_q, d.h_kv, d.d, d.io_dtype)


def gdn_attn_commit(d: AttnDims, cache, table, ctx, k, v, path, path_len, new_len, offsets=None, layer=0,
                    stream=None) -> None:
    """Enqueue the append of the accepted paths' keys and values to the cache (see gdn_attn.h).
    path, path_len: as gdn_tree_commit (ragged: gdn_tree_commit_ragged) writes them."""
    B, io = d.batch, _io_dtype(d)
    off, T = _attn_offsets(offsets, d, k)
    if table.dim() != 2:
        raise ValueError("table: expected [B, width]")
    at = _ints(ctx, (B,), "ctx")
    rows = [_attn_rows(k, T, d.h_kv, d.d, io, "k"), _attn_rows(v, T, d.h_kv, d.d, io, "v")]
    nodes = _ints(path, (B, d.n_nodes) if offsets is None else (T,), "path")
    if T == 0:                                   # trees without nodes: their tensors have no memory, and none is read
        rows, nodes = [AttnRows(at, d.d, d.d)] * 2, at
    _call("gdn_attn_commit", ctypes.byref(d), off, _cache_ref(cache), layer,
          _ints(table, (B, table.shape[1]), "table"), table.shape[1], at, *rows, nodes,
          _ints(path_len, (B,), "path_len"), _ints(new_len, (B,), "new_len"), _stream(stream))


def _page_state(pd, ref, table, held, length):
    return (_ints(ref, (pd.n_pages,), "ref"), _ints(table, (pd.n_slots, pd.width), "table"),
            _ints(held, (pd.n_slots,), "held"), _ints(length, (pd.n_slots,), "length"))


def gdn_pages_fork(pd: PageDims, src_seq, dst_seq, ref, table, held, length, status, stream=None) -> None:
    """Enqueue dst_seq[i] becoming a second holder of src_seq[i]'s pages (see gdn_attn.h)."""
    n = src_seq.numel()
    _call("gdn_pages_fork", ctypes.byref(pd), n, _ints(src_seq, (n,), "src_seq"), _ints(dst_seq, (n,), "dst_seq"),
          *_page_state(pd, ref, table, held, length), _ints(status, (n,), "status"), _stream(stream))


def gdn_pages_reserve(pd: PageDims, need, ref, table, held, length, src, dst, count, status, stream=None) -> None:
    """Enqueue the allocation of need[s] more rows per sequence (see gdn_attn.h); the page copies it
    takes are src, dst, count, for gdn_pages_copy."""
    S = pd.n_slots
    _call("gdn_pages_reserve", ctypes.byref(pd), _ints(need, (S,), "need"),
          *_page_state(pd, ref, table, held, length), _ints(src, (S,), "src"), _ints(dst, (S,), "dst"),
          _ints(count, (1,), "count"), _ints(status, (S,), "status"), _stream(stream))


def gdn_pages_copy(cache, src, dst, count, stream=None) -> None:
    """Enqueue the copies of pages src[i] to dst[i], i < count, in every layer (see gdn_attn.h)."""
    n = src.numel()
    _call("gdn_pages_copy", _cache_ref(cache), n, _ints(src, (n,), "src"), _ints(dst, (n,), "dst"),
          _ints(count, (1,), "count"), _stream(stream))


def gdn_pages_free(pd: PageDims, drop, ref, table, held, length, stream=None) -> None:
    """Enqueue the return of the pages of every sequence with drop[s] != 0 (see gdn_attn.h)."""
    _call("gdn_pages_free", ctypes.byref(pd), _ints(drop, (pd.n_slots,), "drop"),
          *_page_state(pd, ref, table, held, length), _stream(stream))


def gdn_pages_compact(pd: PageDims, ref, table, held, src, dst, count, remap, stream=None) -> None:
    """Enqueue the move of held pages to the front of the pool: bookkeeping here, data by
    gdn_pages_copy(cache, src, dst, count).  At most src.numel() pages move."""
    n = src.numel()
    _call("gdn_pages_compact", ctypes.byref(pd), n, _ints(ref, (pd.n_pages,), "ref"),
          _ints(table, (pd.n_slots, pd.width), "table"), _ints(held, (pd.n_slots,), "held"),
          _ints(src, (n,), "src"), _ints(dst, (n,), "dst"), _ints(count, (1,), "count"),
          _ints(remap, (pd.n_pages,), "remap"), _stream(stream))
