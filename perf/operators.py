"""Cases for timing the attention-layer operators of a decode step.

Four operators: rotary positions of a draft tree's rows ("rope"), attention of a
draft tree over a paged cache ("attend"), the append of the accepted path's rows
to the cache ("append") and the page bookkeeping with its copies ("pages").
With ``own`` false `run` computes them from elementary torch operations in 32
bits (64 for angles); with ``own`` true it calls this repository's package.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
NEG = float("-inf")


# ---------------------------------------------------------------- cases

def _rope(name, batch, nodes, hq, hkv, d, rot, layout, io, scaling, ctx, ragged=False):
    return dict(name=name, op="rope", batch=batch, nodes=nodes, hq=hq, hkv=hkv, d=d, rot=rot,
                layout=layout, io=io, scaling=scaling, ctx=ctx, ragged=ragged)


def _attend(name, batch, nodes, tree, hq, hkv, d, io, ctx_min, ctx_max, page, order, ragged=False):
    return dict(name=name, op="attend", batch=batch, nodes=nodes, tree=tree, hq=hq, hkv=hkv, d=d,
                io=io, ctx_min=ctx_min, ctx_max=ctx_max, page=page, order=order, ragged=ragged)


def _append(name, batch, nodes, path, hkv, d, io, ctx, page, order):
    return dict(name=name, op="append", batch=batch, nodes=nodes, path=path, hkv=hkv, d=d, io=io,
                ctx=ctx, page=page, order=order)


def _pages(name, kind, prompts, children, ctx, page, layers, hkv, d, io):
    return dict(name=name, op="pages", kind=kind, prompts=prompts, children=children, ctx=ctx,
                page=page, layers=layers, hkv=hkv, d=d, io=io)


def listed():
    return [
        # one sequence, one new token: nothing but latency
        _rope("rope_token_b1_f32", 1, 1, 32, 4, 128, 64, "interleaved", "f32", "none", 4000),
        # the benchmark's batch of 128-node trees, whole heads rotated
        _rope("rope_tree128_b64", 64, 128, 32, 4, 128, 128, "half", "bf16", "none", 8192),
        # draft budgets of different sizes far into a stretched context, a quarter of a wide head
        _rope("rope_ragged_far", 48, 128, 16, 2, 256, 64, "half", "bf16", "parts", 1000000, True),
        # a chat turn's next token for one user
        _attend("attend_token_b1", 1, 1, "token", 16, 4, 128, "bf16", 500, 500, 16, "rows"),
        # next tokens of a full batch with contexts of very different lengths
        _attend("attend_token_b64_long", 64, 1, "token", 32, 4, 128, "bf16", 100, 32768, 16, "rows"),
        # 64-node M = 4 trees (16 query heads), pages that keep each head's rows together
        _attend("attend_tree64_b32", 32, 64, "mary", 16, 4, 128, "bf16", 1500, 4096, 64, "heads"),
        # the benchmark's 128-node M = 8 trees over long contexts
        _attend("attend_tree128_b64", 64, 128, "mary", 32, 4, 128, "bf16", 4096, 8192, 32, "rows"),
        # odd sizes in fp32: random recursive trees, ragged, pages of 24 rows, an empty prefix among them
        _attend("attend_rrt77_f32", 5, 77, "rrt", 8, 4, 64, "f32", 0, 2001, 24, "rows", True),
        # one sequence's accepted path of a 64-node tree
        _append("append_tree64_b1", 1, 64, 17, 4, 128, "bf16", 700, 16, "rows"),
        # a batch's accepted paths
        _append("append_tree128_b64", 64, 128, 16, 8, 128, "bf16", 8192, 32, "heads"),
        # several answers from each cached prompt: fork, room for new rows (the shared last page
        # is copied), and the children dropped again
        _pages("pages_fork_b32x4", "fork", 32, 4, 3000, 16, 8, 4, 128, "bf16"),
        # a pool left in fragments by finished sequences moved together
        _pages("pages_compact", "compact", 96, 0, 6000, 32, 4, 4, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "append", "pages"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "rope":
        batch = _log(rng, 1, 64)
        nodes = rng.choice([1, _log(rng, 2, 128)])
        return _drawn(_rope("", batch, nodes, hkv * rng.choice([1, 2, 4]), hkv, min(d, 128),
                            rng.choice([32, 64]), rng.choice(["half", "interleaved"]), io,
                            rng.choice(["none", "linear", "parts"]), _log(rng, 10, 1000000),
                            rng.random() < 0.5))
    if op == "attend":
        group = rng.choice([1, 2, 4, 8])
        tree = rng.choice(["token", "mary", "rrt", "chain"])
        nodes = 1 if tree == "token" else 8 * rng.randint(1, 16) if tree == "mary" else _log(rng, 2, 300)
        batch = _log(rng, 1, 64)
        # no more products than the largest listed case: 64 x 128 nodes x 32 heads x 8192 x 128
        most = 64 * 128 * 32 * 6144 * 128 // (batch * nodes * hkv * group * d)
        most = min(most if io == "bf16" else most // 16, 2 ** 28 // (batch * hkv * d), 32768)
        ctx = _log(rng, 16, max(32, most))
        return _drawn(_attend("", batch, nodes, tree, hkv * group, hkv, d, io, ctx // rng.choice([1, 2, 50]),
                              ctx, rng.choice([16, 24, 32, 64, 128]), rng.choice(["rows", "heads"]),
                              tree != "token" and rng.random() < 0.4))
    if op == "append":
        nodes = _log(rng, 1, 256)
        return _drawn(_append("", _log(rng, 1, 64), nodes, rng.randint(1, min(nodes, 20)), hkv, d, io,
                              _log(rng, 16, 8192), rng.choice([16, 24, 32, 64]),
                              rng.choice(["rows", "heads"])))
    kind = rng.choice(["fork", "compact"])
    return _drawn(_pages("", kind, _log(rng, 2, 64), rng.randint(1, 4) if kind == "fork" else 0,
                         _log(rng, 20, 4000), rng.choice([16, 24, 32]), rng.randint(1, 4),
                         rng.choice([1, 2, 4]), rng.choice([64, 128]), io))


def _drawn(case):
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _dtype(case):
    return torch.float32 if case["io"] == "f32" else torch.bfloat16


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g, np.random.default_rng(int(seed))


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _frequencies(rot, scaling, theta=10000.0, factor=8.0, original=32768):
    """Radians per position of each rotated pair, float64."""
    f = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    # by parts: fast pairs as they are, slow ones interpolated, a ramp over their turns between
    turns = original * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1.0


def _tree_parents(rng, tree, batch, n):
    """[batch][n] parents, a topological order."""
    p = np.full((batch, n), -1, dtype=np.int64)
    if tree == "chain":
        p[:] = np.arange(-1, n - 1)
    elif tree == "mary":
        width = min(8, n)
        at = np.arange(n)
        level = at // width
        pick = rng.integers(0, width, size=(batch, n))
        p = np.where(level > 0, (level - 1) * width + pick, -1)
    elif tree == "rrt":
        p[:, 1:] = np.floor(rng.random((batch, n - 1)) * np.arange(1, n)).astype(np.int64)
    return p


def _sizes(rng, case):
    """Rows of each sequence: the same ones for every seed, in an order of the seed's own."""
    b, n = case["batch"], case["nodes"]
    if not case.get("ragged"):
        return np.full(b, n, dtype=np.int64)
    fixed = np.random.default_rng(1000 * b + n)
    if case["op"] == "rope" or case["tree"] == "mary":
        sizes = np.minimum(n, 8 * fixed.integers(1, max(1, n // 8) + 1, size=b))
    else:
        sizes = fixed.integers(0, n + 1, size=b)
    sizes[0] = n
    return rng.permutation(sizes)


def _pool(rng, g, case, lengths, most, rows):
    """A paged cache that holds `lengths[b]` of up to `most` rows of each sequence and has room for `rows`
    more: key and value pages of random rows (rows that belong to nobody among them) and the page table."""
    page, dt = case["page"], _dtype(case)
    held = -(-(lengths + rows) // page)
    total, width = int(held.sum()), -(-(most + rows) // page)
    n_pages = len(lengths) * width + 3
    ids = rng.permutation(n_pages)[:total]
    table = np.full((len(lengths), width), -1, dtype=np.int64)
    table[np.arange(width)[None, :] < held[:, None]] = ids
    if case.get("order") == "heads":  # [page][head][row][d] in memory, seen as [page][row][head][d]
        shape = (n_pages, case["hkv"], page, case["d"])
        k, v = (_normal(g, shape, dt).transpose(-3, -2) for _ in range(2))
    else:
        shape = (n_pages, page, case["hkv"], case["d"])
        k, v = (_normal(g, shape, dt) for _ in range(2))
    return k, v, _int32(table)


def _prepare_rope(case, seed):
    g, rng = _gen(seed)
    b, n, hq, hkv, d = (case[x] for x in ("batch", "nodes", "hq", "hkv", "d"))
    sizes = _sizes(rng, case)
    rows = int(sizes.sum())
    fused = _normal(g, (rows, (hq + 2 * hkv), d), _dtype(case))  # one projection's output: q, k, v
    freq, amp = _frequencies(case["rot"], case["scaling"])
    par = _tree_parents(rng, "mary", b, n)
    depth = np.zeros((b, n), dtype=np.int64)
    for i in range(n):
        depth[:, i] = np.where(par[:, i] < 0, 0, depth[np.arange(b), np.maximum(par[:, i], 0)] + 1)
    s = dict(case=case, q=fused[:, :hq], k=fused[:, hq:hq + hkv],
             freq=torch.from_numpy(freq).to(DEV), amp=amp,
             ctx=_int32(rng.integers(case["ctx"] // 2, case["ctx"] + 1, size=b)), depth=_int32(depth),
             q_out=torch.empty((rows, hq, d), dtype=_dtype(case), device=DEV),
             k_out=torch.empty((rows, hkv, d), dtype=_dtype(case), device=DEV),
             offsets=_int32(np.concatenate([[0], np.cumsum(sizes)])) if case["ragged"] else None)
    return s


def _prepare_attend(case, seed):
    g, rng = _gen(seed)
    b, n, hq, hkv, d = (case[x] for x in ("batch", "nodes", "hq", "hkv", "d"))
    sizes = _sizes(rng, case)
    rows = int(sizes.sum())
    lo, hi = case["ctx_min"], case["ctx_max"]
    lengths = rng.integers(lo, hi + 1, size=b)
    if b > 1:
        lengths[:2] = (hi, lo)
    kp, vp, table = _pool(rng, g, case, lengths, hi, n)
    par = _tree_parents(rng, case["tree"], b, n)
    words = (n + 31) // 32
    anc = np.zeros((b, n, words * 32), dtype=bool)
    at = np.arange(b)
    for i in range(n):  # strict ancestors: the parent's and the parent
        has = par[:, i] >= 0
        p = np.maximum(par[:, i], 0)
        anc[:, i] = anc[at, p] & has[:, None]
        anc[at[has], i, p[has]] = True
    anc &= (np.arange(n)[None, :] < sizes[:, None])[:, :, None]
    bits = np.packbits(anc, axis=-1, bitorder="little").view(np.uint32).view(np.int32)
    dt = _dtype(case)
    # scores of a standard deviation of two: some keys matter, most hardly do
    q = _normal(g, (rows, hq, d), dt, 2.0)
    fused = _normal(g, (rows, 2 * hkv, d), dt)
    return dict(case=case, q=q, k=fused[:, :hkv], v=fused[:, hkv:], kp=kp, vp=vp, table=table,
                ctx=_int32(lengths), anc=torch.from_numpy(np.ascontiguousarray(bits)).to(DEV),
                status=torch.zeros(b, dtype=torch.int32, device=DEV), scale=d ** -0.5,
                o=torch.empty((rows, hq, d), dtype=dt, device=DEV),
                offsets=_int32(np.concatenate([[0], np.cumsum(sizes)])) if case["ragged"] else None)


def _prepare_append(case, seed):
    g, rng = _gen(seed)
    b, n, hkv, d, most = (case[x] for x in ("batch", "nodes", "hkv", "d", "path"))
    lengths = rng.integers(case["ctx"] // 2, case["ctx"] + 1, size=b)
    kp, vp, table = _pool(rng, g, case, lengths, case["ctx"], n)
    taken = rng.integers(0, most + 1, size=b)
    taken[0] = most
    path = np.full((b, n), -1, dtype=np.int64)
    for i in range(b):
        path[i, :taken[i]] = np.sort(rng.permutation(n)[:taken[i]])
    fused = _normal(g, (b * n, 2 * hkv, d), _dtype(case))
    return dict(case=case, k=fused[:, :hkv], v=fused[:, hkv:], kp=kp, vp=vp, table=table,
                ctx=_int32(lengths), path=_int32(path), path_len=_int32(taken),
                new_len=torch.empty(b, dtype=torch.int32, device=DEV))


def _prepare_pages(case, seed):
    g, rng = _gen(seed)
    prompts, page, layers = case["prompts"], case["page"], case["layers"]
    lengths = rng.integers(max(1, case["ctx"] // 4), case["ctx"] + 1, size=prompts)
    if case["kind"] == "fork":
        # prompts in the first slots, room for the children's new rows in the pool
        slots = prompts * (1 + case["children"])
        spare = prompts * case["children"] * 3
        full = np.concatenate([lengths, np.zeros(slots - prompts, dtype=np.int64)])
    else:
        slots, spare, full = prompts, 0, lengths
    held = -(-full // page)
    total = int(held.sum())
    width = -(-case["ctx"] // page) + 2
    n_pages = prompts * (width - 2) + spare + 5
    ids = rng.permutation(n_pages)[:total]
    table = np.full((slots, width), -1, dtype=np.int64)
    table[np.arange(width)[None, :] < held[:, None]] = ids
    if case["kind"] == "compact":  # every third sequence is done: its pages are holes
        done = np.arange(slots) % 3 == 1
        table[done], held[done], full[done] = -1, 0, 0
    ref = np.zeros(n_pages, dtype=np.int64)
    ref[table[table >= 0]] = 1
    shape = (layers, n_pages, page, case["hkv"], case["d"])
    kp, vp = (_normal(g, shape, _dtype(case)) for _ in range(2))
    s = dict(case=case, kp=kp, vp=vp, table=_int32(table), ref=_int32(ref), held=_int32(held),
             length=_int32(full), n_pages=n_pages, slots=slots, width=width)
    empty = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    if case["kind"] == "fork":
        n = slots - prompts
        s.update(src_seq=_int32(np.arange(n) % prompts), dst_seq=_int32(np.arange(prompts, slots)),
                 need=_int32(np.where(np.arange(slots) < prompts, 0, rng.integers(1, page + 1, size=slots))),
                 drop=_int32(np.arange(slots) >= prompts), fork_status=empty(n), status=empty(slots),
                 src=empty(slots), dst=empty(slots), count=empty(1))
    else:
        live = int(held.sum())
        moves = max(1, int((np.nonzero(ref)[0] >= live).sum()))
        s.update(table0=s["table"].clone(), ref0=s["ref"].clone(), src=empty(moves), dst=empty(moves),
                 count=empty(1), remap=empty(n_pages))
    return s


def prepare(case, seed):
    return {"rope": _prepare_rope, "attend": _prepare_attend, "append": _prepare_append,
            "pages": _prepare_pages}[case["op"]](case, seed)


# ---------------------------------------------------------------- the package's operators

def _own_rope(s):
    import tree_masked_gated_amd as T
    c = s["case"]
    if "dims" not in s:
        s["dims"] = T.attn_dims(c["batch"], c["nodes"], c["hq"], c["hkv"], c["d"], c["io"])
        s["rope"] = T.rope_dims(c["rot"], c["layout"], s["amp"])
    T.gdn_attn_rope(s["dims"], s["rope"], s["q"], s["k"], s["freq"], s["ctx"], s["depth"], s["q_out"],
                    s["k_out"], offsets=s["offsets"])
    return s["q_out"], s["k_out"]


def _own_attend(s):
    import tree_masked_gated_amd as T
    c = s["case"]
    if "dims" not in s:
        s["dims"] = T.attn_dims(c["batch"], c["nodes"], c["hq"], c["hkv"], c["d"], c["io"], s["scale"])
        s["cache"] = T.PagedCache(s["kp"], s["vp"])
        s["workspace"] = T.attn_workspace(s["dims"])
    T.gdn_attn_verify(s["dims"], s["cache"], s["table"], s["ctx"], s["q"], s["k"], s["v"], s["anc"],
                      s["status"], s["o"], s["workspace"], offsets=s["offsets"])
    return s["o"]


def _own_append(s):
    import tree_masked_gated_amd as T
    c = s["case"]
    if "dims" not in s:
        s["dims"] = T.attn_dims(c["batch"], c["nodes"], c["hkv"], c["hkv"], c["d"], c["io"])
        s["cache"] = T.PagedCache(s["kp"], s["vp"])
    T.gdn_attn_commit(s["dims"], s["cache"], s["table"], s["ctx"], s["k"], s["v"], s["path"],
                      s["path_len"], new_len=s["new_len"])
    return s["kp"], s["vp"], s["new_len"]


def _own_pages(s):
    import tree_masked_gated_amd as T
    c = s["case"]
    if "dims" not in s:
        s["dims"] = T.page_dims(s["n_pages"], c["page"], s["slots"], s["width"])
        s["cache"] = T.PagedCache(s["kp"], s["vp"])
    if c["kind"] == "compact":
        s["table"].copy_(s["table0"])
        s["ref"].copy_(s["ref0"])
        T.gdn_pages_compact(s["dims"], s["ref"], s["table"], s["held"], s["src"], s["dst"], s["count"],
                            s["remap"])
        T.gdn_pages_copy(s["cache"], s["src"], s["dst"], s["count"])
        return s["kp"], s["vp"], s["table"], s["ref"], s["count"]
    T.gdn_pages_fork(s["dims"], s["src_seq"], s["dst_seq"], s["ref"], s["table"], s["held"], s["length"],
                     s["fork_status"])
    T.gdn_pages_reserve(s["dims"], s["need"], s["ref"], s["table"], s["held"], s["length"], s["src"],
                        s["dst"], s["count"], s["status"])
    T.gdn_pages_copy(s["cache"], s["src"], s["dst"], s["count"])
    forked = s["table"].clone()
    T.gdn_pages_free(s["dims"], s["drop"], s["ref"], s["table"], s["held"], s["length"])
    return (s["kp"], s["vp"], forked, s["table"], s["ref"], s["held"], s["length"], s["count"],
            s["fork_status"], s["status"])


# ---------------------------------------------------------------- plain forms

def _row_map(offsets, rows):
    """Sequence and node index of each packed row."""
    at = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(offsets.long(), at, right=True) - 1
    return seq, at - offsets.long()[seq]


def _plain_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    pos = s["ctx"].long()[:, None] + s["depth"].long()
    pos = pos.reshape(-1) if s["offsets"] is None else pos[_row_map(s["offsets"], s["q"].shape[0])]
    angle = pos.double()[:, None] * s["freq"]
    cos = (torch.cos(angle) * s["amp"]).float()[:, None, :]
    sin = (torch.sin(angle) * s["amp"]).float()[:, None, :]

    def turn(x):
        x32 = x.float()
        if c["layout"] == "half":
            a, b = x32[..., :half], x32[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        return torch.cat([y, x32[..., rot:]], dim=-1).to(x.dtype)

    s["q_out"].copy_(turn(s["q"]))
    s["k_out"].copy_(turn(s["k"]))
    return s["q_out"], s["k_out"]


def _plain_attend(s):
    c = s["case"]
    b, n, hq, hkv, d, page = (c[x] for x in ("batch", "nodes", "hq", "hkv", "d", "page"))
    group, most = hq // hkv, c["ctx_max"]
    pages = min(-(-most // page), s["table"].shape[1])
    idx = s["table"][:, :pages].long().clamp(min=0)
    off = s["offsets"]
    if off is None:
        seq = node = None
        dense = lambda x: x.reshape(b, n, *x.shape[1:])  # noqa: E731
    else:
        seq, node = _row_map(off, s["q"].shape[0])
        dense = lambda x: x.new_zeros(b, n, *x.shape[1:]).index_put_((seq, node), x)  # noqa: E731
    # [b, hkv, keys, d]: the prefix's rows, then the tree's
    gather = lambda p, t: torch.cat([p[idx].reshape(b, -1, hkv, d).float(),  # noqa: E731
                                     dense(t).float()], dim=1).transpose(1, 2).contiguous()
    keys, values = gather(s["kp"], s["k"]), gather(s["vp"], s["v"])
    word = torch.arange(n, device=DEV)
    tree = (s["anc"].long()[:, :, word // 32] >> (word % 32)) & 1
    tree = (tree == 1) | torch.eye(n, dtype=torch.bool, device=DEV)
    prefix = torch.arange(pages * page, device=DEV)[None, :] < s["ctx"].long()[:, None]
    seen = torch.cat([prefix[:, None, :].expand(-1, n, -1), tree], dim=2)
    q = dense(s["q"]).float().reshape(b, n, hkv, group, d).transpose(1, 2).reshape(b, hkv, n * group, d)
    scores = torch.matmul(q, keys.transpose(2, 3).contiguous()) * s["scale"]
    scores = scores.reshape(b, hkv, n, group, -1).masked_fill_(~seen[:, None, :, None, :], NEG)
    weight = torch.exp(scores - scores.amax(-1, keepdim=True))
    total = weight.sum(-1, keepdim=True)
    o = torch.matmul(weight.reshape(b, hkv, n * group, -1), values).reshape(b, hkv, n, group, d) / total
    o = o.transpose(1, 2).reshape(b, n, hq, d).to(s["o"].dtype)
    s["o"].copy_(o.reshape(-1, hq, d) if off is None else o[seq, node])
    return s["o"]


def _plain_append(s):
    c = s["case"]
    b, n, page = c["batch"], c["nodes"], c["page"]
    step = torch.arange(n, device=DEV)
    real = (step[None, :] < s["path_len"].long()[:, None])[..., None, None]
    node = s["path"].long().clamp(min=0) + (torch.arange(b, device=DEV) * n)[:, None]
    at = s["ctx"].long()[:, None] + step[None, :]
    pid = torch.gather(s["table"].long(), 1, at // page)
    where = (pid, at % page)
    s["kp"][where] = torch.where(real, s["k"][node], s["kp"][where])
    s["vp"][where] = torch.where(real, s["v"][node], s["vp"][where])
    s["new_len"].copy_(s["ctx"] + s["path_len"].clamp(min=0))
    return s["kp"], s["vp"], s["new_len"]


def _copy_pages(s, src, dst, real):
    """Page src[i] over page dst[i] where real[i]; elsewhere dst[i] is a page of its own and stays."""
    source = torch.where(real, src, dst)
    s["kp"][:, dst] = s["kp"][:, source]
    s["vp"][:, dst] = s["vp"][:, source]


def _plain_fork(s):
    page, slots, width = s["case"]["page"], s["slots"], s["width"]
    table, ref, held, length = s["table"], s["ref"], s["held"], s["length"]
    col = torch.arange(width, device=DEV)
    # children share the prompt's pages
    f, t = s["src_seq"].long(), s["dst_seq"].long()
    used = -(-length[f] // page)
    mine = col[None, :] < used[:, None]
    rows = table[f]
    table[t] = torch.where(mine, rows, -1)
    ref.index_add_(0, rows.clamp(min=0).reshape(-1).long(), mine.reshape(-1).int())
    held[t], length[t] = used, length[f]
    s["fork_status"].zero_()
    # room for the new rows: missing pages, and a page of its own for a shared last one
    need, at = s["need"], torch.arange(slots, device=DEV)
    wants = need > 0
    want = -(-(length + need) // page)
    tail = (length // page).long()
    part = wants & (length % page > 0)
    tail_page = torch.gather(table.long(), 1, tail.clamp(max=width - 1)[:, None])[:, 0]
    shares = part & (ref[tail_page.clamp(min=0)] > 1)
    same = (tail_page[:, None] == tail_page[None, :]) & shares[:, None] & shares[None, :]
    later = (same & (at[None, :] > at[:, None])).any(1)
    everyone = same.sum(1) == ref[tail_page.clamp(min=0)]
    copies = shares & ~(everyone & ~later)
    fits = wants & (want <= width)
    demand = torch.where(fits, (want - held).clamp(min=0) + copies, 0)
    upto = torch.cumsum(demand, 0)
    order = torch.argsort((ref > 0).int(), stable=True)
    enough = upto <= (ref == 0).sum()
    good = fits & (enough | (demand == 0) & ~shares)
    s["status"].copy_(torch.where(~wants | good, 0, torch.where(fits, -2, -1)))
    copies &= good
    first = upto - demand
    fresh = good[:, None] & (col[None, :] >= held[:, None]) & (col[None, :] < want[:, None])
    slot = torch.where(fresh, (first + copies)[:, None] + col[None, :] - held[:, None], first[:, None])
    own_tail = copies[:, None] & (col[None, :] == tail[:, None])
    new = fresh | own_tail
    pick = order[slot.clamp(0, len(order) - 1)]
    ref.index_add_(0, pick.reshape(-1), new.reshape(-1).int())
    ref.index_add_(0, tail_page.clamp(min=0), -copies.int())
    table.copy_(torch.where(new, pick.int(), table))
    held.copy_(torch.where(good, torch.maximum(want, held), held))
    s["count"].copy_(copies.sum(0, keepdim=True))
    # the copies; a sequence without one keeps a page that no other sequence names here
    _copy_pages(s, tail_page, torch.where(copies, order[first.clamp(0, len(order) - 1)],
                                          order[len(order) - 1 - at]), copies)
    forked = table.clone()
    # the children are done
    gone = s["drop"][:, None].bool() & (col[None, :] < held[:, None])
    ref.index_add_(0, table.clamp(min=0).reshape(-1).long(), -gone.reshape(-1).int())
    table.masked_fill_(s["drop"][:, None].bool(), -1)
    held.masked_fill_(s["drop"].bool(), 0)
    length.masked_fill_(s["drop"].bool(), 0)
    return (s["kp"], s["vp"], forked, table, ref, held, length, s["count"], s["fork_status"], s["status"])


def _plain_compact(s):
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    table, ref, n = s["table"], s["ref"], s["n_pages"]
    at = torch.arange(n, device=DEV)
    live = ref > 0
    total = live.sum()
    moves, holes = live & (at >= total), ~live & (at < total)
    source = torch.argsort((~moves).int(), stable=True)
    target = torch.argsort((~holes).int(), stable=True)
    real = at < moves.sum()
    remap = at.clone()
    remap[source] = torch.where(real, target, source)
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()].int(), table))
    came = at.clone()
    came[target] = torch.where(real, source, target)
    ref.copy_(torch.where(at < total, ref[came], 0))
    m = len(s["src"])
    _copy_pages(s, source[:m], target[:m], real[:m])
    s["count"].copy_(moves.sum().reshape(1))
    return s["kp"], s["vp"], table, ref, s["count"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "attend": _own_attend, "append": _own_append,
                "pages": _own_pages}[op](state)
    if op == "pages":
        return (_plain_compact if state["case"]["kind"] == "compact" else _plain_fork)(state)
    return {"rope": _plain_rope, "attend": _plain_attend, "append": _plain_append}[op](state)


# ---------------------------------------------------------------- bytes and operations

def work(case):
    e = 4 if case["io"] == "f32" else 2
    rng = np.random.default_rng(1)
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "pages":
        page_bytes = 2 * case["layers"] * case["page"] * hkv * d * e
        if case["kind"] == "fork":
            n = case["prompts"] * case["children"]
            entries = n * case["ctx"] * 5 // 8 // case["page"]
            return {"bytes": 2 * n * page_bytes + 20 * entries, "flops": entries}
        pages = case["prompts"] * (case["ctx"] * 5 // 8 // case["page"] + 1)
        return {"bytes": 2 * page_bytes * pages * 2 // 9 + 16 * pages, "flops": pages}
    b, n = case["batch"], case["nodes"]
    if case["op"] == "append":
        rows = b * (case["path"] + 1) / 2
        return {"bytes": 4 * rows * hkv * d * e + 8 * rows, "flops": rows}
    hq = case["hq"]
    rows = float(_sizes(rng, case).sum())
    if case["op"] == "rope":
        heads = hq + hkv
        return {"bytes": rows * (2 * heads * d * e + 4) + 8 * case["rot"],
                "flops": rows * heads * case["rot"] * 3}
    ctx = (case["ctx_min"] + case["ctx_max"]) / 2
    per = rows / b
    keys = rows * ctx + rows * min(per, 16)  # a node sees the prefix and its few ancestors
    return {"bytes": 2 * b * ctx * hkv * d * e + rows * (2 * hq + 2 * hkv) * d * e + rows * (n + 31) // 32 * 4
            + 4 * b * ctx / case["page"], "flops": 4 * keys * hq * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    b, n = case.get("batch"), case.get("nodes")
    if case["op"] in ("rope", "attend", "append"):
        lens = [n] * b if s.get("offsets") is None else torch.diff(s["offsets"]).tolist()
        starts = np.concatenate([[0], np.cumsum(lens)]).astype(int)
    if case["op"] == "rope":
        rot, out = case["rot"], []
        turns = torch.cat([s["ctx"][i].double() + s["depth"][i, :lens[i]].double() for i in range(b)])
        phase = torch.polar(torch.full_like(s["freq"], s["amp"]).expand(len(turns), -1).contiguous(),
                            turns[:, None] * s["freq"])[:, None, :]
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            if case["layout"] == "half":
                z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * phase
                y[..., :rot] = torch.cat([z.real, z.imag], -1)
            else:
                z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], -1, 2).contiguous()) * phase
                y[..., :rot] = torch.view_as_real(z).flatten(-2)
            out.append(y)
        return tuple(out)
    if case["op"] == "attend":
        group, out = case["hq"] // case["hkv"], []
        bits = np.unpackbits(s["anc"].cpu().numpy().view(np.uint8), axis=-1, bitorder="little")
        for i in range(b):
            m, length = lens[i], int(s["ctx"][i])
            if m == 0:
                continue
            ids = s["table"][i, :-(-length // case["page"])].long()
            own_rows = slice(starts[i], starts[i] + m)
            cat = lambda p, t: torch.cat([p[ids].flatten(0, 1)[:length].double(),  # noqa: E731
                                          t[own_rows].double()])
            keys, values = cat(s["kp"], s["k"]), cat(s["vp"], s["v"])
            look = torch.ones(m, length + m, dtype=torch.bool, device=DEV)
            look[:, length:] = torch.from_numpy(bits[i, :m, :m].astype(bool) | np.eye(m, dtype=bool)).to(DEV)
            q = s["q"][own_rows].double()
            o = torch.empty_like(q)
            for h in range(case["hkv"]):
                mine = q[:, h * group:(h + 1) * group].permute(1, 0, 2).contiguous()
                sc = (mine.reshape(group * m, -1) @ keys[:, h].T.contiguous()).reshape(group, m, -1) * s["scale"]
                p = torch.softmax(sc.masked_fill(~look, NEG), -1)
                o[:, h * group:(h + 1) * group] = (p.reshape(group * m, -1) @ values[:, h]).reshape(
                    group, m, -1).permute(1, 0, 2)
            out.append(o)
        return torch.cat(out)
    if case["op"] == "append":
        pools = [s["kp"].double().clone(), s["vp"].double().clone()]
        path, taken, ctx, table = (s[x].tolist() for x in ("path", "path_len", "ctx", "table"))
        for i in range(b):
            for j in range(taken[i]):
                pid, row = table[i][(ctx[i] + j) // case["page"]], (ctx[i] + j) % case["page"]
                for pool, new in zip(pools, (s["k"], s["v"])):
                    pool[pid, row] = new[i * n + path[i][j]].double()
        return (*pools, None)
    # pages: the bookkeeping one sequence and one page after the other, the data moved accordingly
    pools = [s["kp"].double().clone(), s["vp"].double().clone()]
    table, ref, held, length = (s[x].tolist() for x in ("table", "ref", "held", "length"))
    page = case["page"]
    if case["kind"] == "compact":
        total = sum(r > 0 for r in ref)
        holes = [p for p in range(total) if ref[p] == 0]
        for hole, p in zip(holes, [p for p in range(total, len(ref)) if ref[p] > 0]):
            for pool in pools:
                pool[:, hole] = pool[:, p]
        return (*pools, None, None, None)
    for f, t in zip(s["src_seq"].tolist(), s["dst_seq"].tolist()):
        length[t] = length[f]
        for c in range(-(-length[f] // page)):
            table[t][c] = table[f][c]
            ref[table[f][c]] += 1
    free = [p for p, r in enumerate(ref) if r == 0]
    for i, more in enumerate(s["need"].tolist()):
        if more == 0:
            continue
        c = length[i] // page
        old = table[i][c]
        if length[i] % page and ref[old] > 1:
            table[i][c] = free.pop(0)
            ref[old] -= 1
            for pool in pools:
                pool[:, table[i][c]] = pool[:, old]
        for c in range(-(-length[i] // page), -(-(length[i] + more) // page)):
            table[i][c] = free.pop(0)
    return (*pools, *[None] * 8)
