"""Cases for timing the gated delta rule over whole sequences and the scores of tokens.

Five operators: the gated delta rule over ragged sequences ("forward"), its gradients ("backward"),
its step by one token on a pool of states ("step"), log-probabilities of given tokens with entropy and
top alternatives ("scores") and their gradient ("scores_grad").  With ``own`` false `run` computes them
from elementary torch operations in 32 bits (64 for running sums of logarithms); with ``own`` true it
calls this repository's package.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
CHUNK = 64


# ---------------------------------------------------------------- cases

def _rule(name, op, batch, rows, hk, hv, dk, dv, io, prior):
    """rows: the longest sequence's; prior: whether the sequences have a state before them."""
    return dict(name=name, op=op, batch=batch, rows=rows, hk=hk, hv=hv, dk=dk, dv=dv, io=io, prior=prior)


def _step(name, batch, slots, hk, hv, dk, dv, io):
    return dict(name=name, op="step", batch=batch, slots=slots, hk=hk, hv=hv, dk=dk, dv=dv, io=io)


def _scores(name, op, rows, vocab, pad, topk, io):
    """pad: entries at the end of the vocabulary that are no tokens (their logits are -inf)."""
    return dict(name=name, op=op, rows=rows, vocab=vocab, pad=pad, topk=topk, io=io)


def listed():
    return [
        # one long prompt through a layer of the benchmark's head layout
        _rule("forward_prompt_b1", "forward", 1, 8192, 16, 32, 128, 128, "bf16", False),
        # a batch of prompts and of later pieces of prompts, lengths all different
        _rule("forward_ragged_b24", "forward", 24, 2048, 16, 32, 128, 128, "bf16", True),
        # small heads in fp32, a few short sequences
        _rule("forward_short_f32", "forward", 3, 100, 2, 4, 64, 64, "f32", True),
        # a training batch of the same layer
        _rule("backward_train_b4", "backward", 4, 2048, 16, 32, 128, 128, "bf16", False),
        # gradients through a given state, odd head sizes in fp32
        _rule("backward_odd_f32", "backward", 5, 333, 2, 4, 48, 80, "f32", True),
        # one user's next token, and a full batch's out of a larger pool of states
        _step("step_b1", 1, 1, 16, 32, 128, 128, "bf16"),
        _step("step_b64", 64, 96, 16, 32, 128, 128, "bf16"),
        # the drafter's alternatives after one prefix: latency
        _scores("scores_draft_b1", "scores", 1, 32000, 0, 8, "bf16"),
        # the verifier's tokens after every node of the benchmark's trees
        _scores("scores_tree128_b64", "scores", 8192, 65536, 0, 1, "bf16"),
        # many alternatives over an odd vocabulary with padding, fp32
        _scores("scores_wide_f32", "scores", 300, 50001, 81, 64, "f32"),
        # the drafter's loss on a batch: given tokens and the verifier's alternatives
        _scores("scores_grad_train", "scores_grad", 4096, 65536, 0, 8, "bf16"),
        # a few rows over an odd vocabulary
        _scores("scores_grad_odd_f32", "scores_grad", 33, 10007, 7, 0, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "step", "scores", "scores_grad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scores", "scores_grad"):
        vocab = _log(rng, 500, 150000)
        most = (2 ** 29 if op == "scores" else 2 ** 28) // vocab // (1 if io == "bf16" else 2)
        rows = _log(rng, 1, min(8192, most))
        topk = rng.choice([0, 1, 1, 4, 8, 20, 64])
        return _drawn(_scores("", op, rows, vocab, rng.choice([0, 0, _log(rng, 1, 100)]), topk, io))
    hk = rng.choice([1, 2, 4, 8, 16])
    hv = hk * rng.choice([1, 2, 2, 4])
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64), (48, 80), (256, 256), (96, 33)])
    if op == "step":
        batch = _log(rng, 1, max(1, min(128, 64 * 32 * 128 * 128 // (hv * dk * dv))))
        return _drawn(_step("", batch, batch + rng.choice([0, batch // 2, 3]), hk, hv, dk, dv, io))
    # no more products than the largest listed case of the kind, and no longer a sequence
    most = (24 * 1100 if op == "forward" else 4 * 1900) * 32 * 128 * 128 // (hv * dk * dv)
    most //= 1 if io == "bf16" else 4
    batch = _log(rng, 1, 32)
    rows = _log(rng, 1, max(2, min(8192 if op == "forward" else 2048, most // batch)))
    return _drawn(_rule("", op, batch, rows, hk, hv, dk, dv, io, rng.random() < 0.5))


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


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _lengths(rng, case):
    """Rows of each sequence: the same ones for every seed, in an order of the seed's own."""
    b, n = case["batch"], case["rows"]
    fixed = np.random.default_rng(1000 * b + n)
    sizes = fixed.integers(n // 2 if case["op"] == "backward" else 0, n + 1, size=b)
    sizes[0] = n
    return rng.permutation(sizes)


def _layer(g, case, rows):
    """Queries, keys and values as slices of one projection's output where heads are equally wide, and gates."""
    hk, hv, dk, dv = (case[x] for x in ("hk", "hv", "dk", "dv"))
    dt = _dtype(case)
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    q = unit(_normal(g, rows, hk, dk)) * dk ** -0.5
    k = unit(_normal(g, rows, hk, dk) + 0.5 * _normal(g, 1, hk, dk))  # keys with a common direction
    v = _normal(g, rows, hv, dv)
    if dk == dv:
        fused = torch.cat([q, k, v], 1).to(dt)
        q, k, v = fused[:, :hk], fused[:, hk:2 * hk], fused[:, 2 * hk:]
    else:
        q, k, v = q.to(dt), k.to(dt), v.to(dt)
    beta = torch.sigmoid(_normal(g, rows, hv))
    # heads that forget within a few rows and heads that remember thousands
    rate = torch.exp(torch.linspace(math.log(1e-3), math.log(0.7), hv, device=DEV))
    gate = torch.exp(-rate * torch.nn.functional.softplus(_normal(g, rows, hv)))
    return dict(q=q, k=k, v=v, beta=beta, g=gate)


def _prepare_rule(case, seed):
    g, rng = _gen(seed)
    sizes = _lengths(rng, case)
    rows, (b, hv, dk, dv) = int(sizes.sum()), (case[x] for x in ("batch", "hv", "dk", "dv"))
    s = dict(case=case, rows=rows, longest=int(sizes.max()), **_layer(g, case, rows),
             offsets=_int32(np.concatenate([[0], np.cumsum(sizes)])))
    s["S0"] = 0.3 * _normal(g, b, hv, dv, dk) if case["prior"] else None
    state = lambda: torch.empty((b, hv, dv, dk), dtype=torch.float32, device=DEV)  # noqa: E731
    like = lambda x: torch.empty(x.shape, dtype=x.dtype, device=DEV)  # noqa: E731
    if case["op"] == "forward":
        s.update(o=like(s["v"]), S_out=state())
    else:
        s.update(d_o=_normal(g, rows, hv, dv).to(_dtype(case)),
                 dS_out=0.1 * _normal(g, b, hv, dv, dk) if case["prior"] else None,
                 dq=like(s["q"]), dk=like(s["k"]), dv=like(s["v"]), dbeta=like(s["beta"]), dlog_g=like(s["g"]),
                 dS0=state() if case["prior"] else None)
    return s


def _prepare_step(case, seed):
    g, rng = _gen(seed)
    b, hv, dk, dv = (case[x] for x in ("batch", "hv", "dk", "dv"))
    s = dict(case=case, **_layer(g, case, b))
    s.update(state=0.3 * _normal(g, case["slots"], hv, dv, dk), slot=_int32(rng.permutation(case["slots"])[:b]),
             o=torch.empty((b, hv, dv), dtype=_dtype(case), device=DEV))
    return s


def _prepare_scores(case, seed):
    g, rng = _gen(seed)
    rows, vocab, real, dt = case["rows"], case["vocab"], case["vocab"] - case["pad"], _dtype(case)
    x = _normal(g, rows, vocab) * 2.5
    x[:, real:] = -math.inf
    # in half of the rows one token stands out, as where a model is sure
    sure = torch.randint(0, real, (rows,), generator=g, device=DEV)
    x[torch.arange(0, rows, 2, device=DEV), sure[::2]] = 14.0
    x = x.to(dt)
    pick = torch.randint(0, real, (rows,), generator=g, device=DEV)
    tokens = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.5, sure, pick).to(torch.int32)
    vec = lambda: torch.empty(rows, dtype=torch.float32, device=DEV)  # noqa: E731
    s = dict(case=case, logits=x, tokens=tokens, logp=vec(), entropy=vec(), lse=vec())
    k = case["topk"]
    if case["op"] == "scores":
        if k:
            s.update(top_logp=torch.empty((rows, k), dtype=torch.float32, device=DEV),
                     top_tok=torch.empty((rows, k), dtype=torch.int32, device=DEV))
        return s
    # what the forward pass left
    y = x.double() if rows * vocab < 2 ** 24 else x.float()
    m = y.amax(1)
    e = torch.exp(y - m[:, None])
    total = e.sum(1)
    mean = torch.where(e > 0, e * (y - m[:, None]), torch.zeros((), dtype=y.dtype, device=DEV)).sum(1) / total
    s["lse"], s["entropy"] = (m + total.log()).float(), (total.log() - mean).float()
    s.update(d_logp=_normal(g, rows), d_entropy=0.1 * _normal(g, rows), d_logits=torch.empty_like(x))
    if k:
        # alternatives of another model's choosing: any distinct tokens
        start = torch.randint(0, real, (rows, 1), generator=g, device=DEV)
        s.update(top_tok=((start + torch.arange(k, device=DEV) * (real // k)) % real).to(torch.int32),
                 d_top_logp=0.3 * _normal(g, rows, k))
    return s


def prepare(case, seed):
    if case["op"] in ("forward", "backward"):
        return _prepare_rule(case, seed)
    return _prepare_step(case, seed) if case["op"] == "step" else _prepare_scores(case, seed)


# ---------------------------------------------------------------- the package's operators

def _own_dims(s):
    import tree_masked_gated_amd as T
    c = s["case"]
    if "dims" not in s:
        s["dims"] = T.rule_dims(c["batch"], c["hk"], c["hv"], c["dk"], c["dv"], c["io"])
        if c["op"] != "step":
            s["ws"] = T.rule_workspace(s["dims"], s["rows"], backward=c["op"] == "backward")
    return T


def _own_forward(s):
    T = _own_dims(s)
    T.gdn_rule_forward(s["dims"], s["offsets"], s["q"], s["k"], s["v"], s["beta"], s["g"], s["o"], s["ws"],
                       S0=s["S0"], S_out=s["S_out"])
    return dict(o=s["o"], S_out=s["S_out"])


GRADS = ("dq", "dk", "dv", "dbeta", "dlog_g", "dS0")


def _own_backward(s):
    T = _own_dims(s)
    T.gdn_rule_backward(s["dims"], s["offsets"], s["q"], s["k"], s["v"], s["beta"], s["g"], s["d_o"], s["dq"],
                        s["dk"], s["dv"], s["dbeta"], s["dlog_g"], s["ws"], S0=s["S0"], dS_out=s["dS_out"],
                        dS0=s["dS0"])
    return {x: s[x] for x in GRADS}


def _own_step(s):
    T = _own_dims(s)
    T.gdn_rule_step(s["dims"], s["q"], s["k"], s["v"], s["beta"], s["g"], s["state"], s["o"], slot=s["slot"])
    return dict(o=s["o"], state=s["state"])


def _own_scores(s):
    import tree_masked_gated_amd as T
    c = s["case"]
    if "dims" not in s:
        s["dims"] = T.score_dims(c["rows"], c["vocab"], c["topk"], c["io"])
        s["ws"] = T.score_workspace(s["dims"])
    T.gdn_token_scores(s["dims"], s["logits"], s["tokens"], s["logp"], s["entropy"], s["lse"], s["ws"],
                       top_logp=s.get("top_logp"), top_tok=s.get("top_tok"))
    return {x: s[x] for x in ("logp", "entropy", "lse", "top_logp", "top_tok") if x in s}


def _own_scores_grad(s):
    import tree_masked_gated_amd as T
    c = s["case"]
    if "dims" not in s:
        s["dims"] = T.score_dims(c["rows"], c["vocab"], c["topk"], c["io"])
    T.gdn_token_scores_backward(s["dims"], s["logits"], s["tokens"], s["lse"], s["entropy"], s["d_logp"],
                                s["d_entropy"], s["d_logits"], top_tok=s.get("top_tok"),
                                d_top_logp=s.get("d_top_logp"))
    return s["d_logits"]


# ---------------------------------------------------------------- the plain forms

class _Chunks:
    """The rows of every sequence in chunks of CHUNK, [batch, value head, chunk, row, ...], padded with rows that
    change nothing; and the parts of the chunked rule that need no state."""

    def __init__(self, s):
        c = s["case"]
        off = s["offsets"].long()
        self.n = max(1, -(-s["longest"] // CHUNK))
        at = torch.arange(self.n * CHUNK, device=DEV)
        self.live = at < (off[1:] - off[:-1])[:, None]
        self.idx = torch.where(self.live, off[:-1, None] + at, 0)
        self.group = c["hv"] // c["hk"]
        self.q, self.k = (self.rows(s[x]).repeat_interleave(self.group, 1) for x in ("q", "k"))
        self.v = self.rows(s["v"])
        self.beta = self.rows(s["beta"][..., None])
        gamma = self.rows(torch.log(s["g"].double())[..., None], torch.float64).cumsum(3)
        self.a = torch.exp(gamma).float()
        self.to_end = torch.exp(gamma[..., -1:, :] - gamma).float()
        low = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=DEV).tril()
        diff = torch.where(low, gamma - gamma.transpose(-1, -2), torch.full((), -math.inf, device=DEV).double())
        self.decay = torch.exp(diff).float()
        self.gram = self.k @ self.k.transpose(-1, -2)
        x = (self.beta * self.decay * self.gram).tril(-1)
        inv = torch.eye(CHUNK, device=DEV).expand_as(x).clone()
        for i in range(1, CHUNK):
            inv[..., i, :i] = -(x[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
        self.inv = inv
        self.y = self.decay * (self.q @ self.k.transpose(-1, -2))

    def rows(self, x, dtype=torch.float32):
        y = torch.where(self.live[..., None, None], x[self.idx].to(dtype), 0)
        return y.unflatten(1, (self.n, CHUNK)).permute(0, 3, 1, 2, 4).contiguous()

    def out(self, x, to):
        """[batch, head, chunk, row, ...] into the packed rows of `to`, heads summed over those that share one."""
        y = x.permute(0, 2, 3, 1, 4).flatten(1, 2)
        if y.shape[2] != to.shape[1]:
            y = y.unflatten(2, (to.shape[1], -1)).sum(3)
        to[self.idx[self.live]] = y[self.live].reshape(-1, *to.shape[1:]).to(to.dtype)
        return to

    def forward(self, S0):
        """Start states [d_k, d_v] of all chunks and the end's, and the pre-write differences and writes."""
        b, hv, _, _, dk = self.k.shape
        h = [torch.zeros((b, hv, dk, self.v.shape[-1]), device=DEV) if S0 is None else S0.transpose(-1, -2)]
        u = []
        for c in range(self.n):
            r = self.beta[:, :, c] * (self.v[:, :, c] - self.a[:, :, c] * (self.k[:, :, c] @ h[-1]))
            u.append(self.inv[:, :, c] @ r)
            h.append(self.a[:, :, c, -1:] * h[-1] + (self.to_end[:, :, c] * self.k[:, :, c]).transpose(-1, -2) @ u[-1])
        return torch.stack(h, 2), torch.stack(u, 2)


def _plain_forward(s):
    t = _Chunks(s)
    h, u = t.forward(s["S0"])
    o = t.a * (t.q @ h[:, :, :-1]) + t.y @ u
    s["S_out"].copy_(h[:, :, -1].transpose(-1, -2))
    return dict(o=t.out(o, s["o"]), S_out=s["S_out"])


def _plain_backward(s):
    t = _Chunks(s)
    h, u = t.forward(s["S0"])
    start, end = h[:, :, :-1], h[:, :, 1:]
    do = t.rows(s["d_o"])
    T = lambda x: x.transpose(-1, -2)  # noqa: E731
    from_o = T(t.y) @ do
    q_do = T(t.a * t.q) @ do
    dend = torch.zeros_like(start)
    dr = torch.empty_like(u)
    dh = torch.zeros_like(h[:, :, 0]) if s["dS_out"] is None else T(s["dS_out"])
    for c in reversed(range(t.n)):
        dend[:, :, c] = dh
        du = from_o[:, :, c] + t.to_end[:, :, c] * (t.k[:, :, c] @ dh)
        dr[:, :, c] = T(t.inv[:, :, c]) @ du
        dh = t.a[:, :, c, -1:] * dh + q_do[:, :, c] - T(t.a[:, :, c] * t.beta[:, :, c] * t.k[:, :, c]) @ dr[:, :, c]
    dv = t.beta * dr
    low = (t.decay * t.gram).tril(-1)
    w = t.v - t.a * (t.k @ start) - low @ u
    dy = t.decay * (do @ T(u))
    dx = (-t.beta * t.decay * (dr @ T(u))).tril(-1)
    o = t.a * (t.q @ start) + t.y @ u
    dq = t.a * (do @ T(start)) + dy @ t.k
    dk = T(dy) @ t.q + (dx + T(dx)) @ t.k + t.to_end * (u @ T(dend)) - t.beta * t.a * (dr @ T(start))
    change = (o * do - t.v * dv).double().sum(-1, keepdim=True)
    last = (end.double() * dend).sum((-1, -2))[..., None, None]
    dlog_g = last + change.flip(3).cumsum(3).flip(3)
    if s["dS0"] is not None:
        s["dS0"].copy_(T(dh))
    return dict(dq=t.out(dq, s["dq"]), dk=t.out(dk, s["dk"]), dv=t.out(dv, s["dv"]),
                dbeta=t.out((dr * w).sum(-1, keepdim=True), s["dbeta"][..., None])[..., 0],
                dlog_g=t.out(dlog_g, s["dlog_g"][..., None])[..., 0], dS0=s["dS0"])


def _plain_step(s):
    c = s["case"]
    at = s["slot"].long()
    q, k = (s[x].float().repeat_interleave(c["hv"] // c["hk"], 1) for x in ("q", "k"))
    p = s["g"][..., None, None] * s["state"][at]
    w = s["v"].float() - (p @ k[..., None])[..., 0]
    new = p + (s["beta"][..., None] * w)[..., None] * k[..., None, :]
    s["state"][at] = new
    s["o"].copy_((new @ q[..., None])[..., 0])
    return dict(o=s["o"], state=s["state"])


def _plain_scores(s):
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(1)
    log = total.log()
    mean = torch.where(e > 0, e * (x - m), 0).sum(1) / total
    got = dict(logp=x.gather(1, s["tokens"].long()[:, None])[:, 0] - m[:, 0] - log, entropy=log - mean,
               lse=m[:, 0] + log)
    if "top_tok" in s:
        # keys that order by value, then by the lower index
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        keys = (order << 32) | (x.shape[1] - 1 - torch.arange(x.shape[1], device=DEV))
        best = x.shape[1] - 1 - (torch.topk(keys, s["case"]["topk"], dim=1).values & 0xFFFFFFFF)
        got.update(top_logp=x.gather(1, best) - m - log[:, None], top_tok=best.to(torch.int32))
    return got


def _plain_scores_grad(s):
    x = s["logits"].float()
    logp = x - s["lse"][:, None]
    p = torch.exp(logp)
    gl, ge = s["d_logp"][:, None], s["d_entropy"][:, None]
    every = gl if "top_tok" not in s else gl + s["d_top_logp"].sum(1, keepdim=True)
    d = torch.where(p > 0, -p * (every + ge * (logp + s["entropy"][:, None])), 0)
    d.scatter_add_(1, s["tokens"].long()[:, None], gl)
    if "top_tok" in s:
        d.scatter_add_(1, s["top_tok"].long(), s["d_top_logp"])
    s["d_logits"].copy_(d)
    return s["d_logits"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"forward": _own_forward, "backward": _own_backward, "step": _own_step, "scores": _own_scores,
                "scores_grad": _own_scores_grad}[op](state)
    return {"forward": _plain_forward, "backward": _plain_backward, "step": _plain_step, "scores": _plain_scores,
            "scores_grad": _plain_scores_grad}[op](state)


# ---------------------------------------------------------------- 64 bits, by definition

def _token(p, k, v, beta):
    """State after one token, given the decayed one; and the difference that the token writes."""
    w = v - torch.matmul(p, k[..., None])[..., 0]
    return p + (beta[..., None] * w)[..., None] * k[..., None, :], w


def _exact_rule(case, s):
    """The rule token by token over all sequences at once; its gradients token by token from the end."""
    b, hv, dk, dv = (case[x] for x in ("batch", "hv", "dk", "dv"))
    n, back = s["longest"], case["op"] == "backward"
    if back and 8 * n * b * hv * dk * dv > 60e9:
        return None
    off = s["offsets"].tolist()
    share = hv // case["hk"]

    def padded(x):
        out = torch.zeros((b, n) + x.shape[1:], dtype=torch.float64, device=DEV)
        for i in range(b):
            out[i, :off[i + 1] - off[i]] = x[off[i]:off[i + 1]].double()
        return out

    def packed(x, to):
        return torch.cat([x[i, :off[i + 1] - off[i]] for i in range(b)]).reshape(to.shape)

    q, k = (padded(s[x]).repeat_interleave(share, 2) for x in ("q", "k"))
    v, beta, g = padded(s["v"]), padded(s["beta"]), padded(s["g"])
    for i in range(b):
        g[i, off[i + 1] - off[i]:] = 1.0
    S = torch.zeros((b, hv, dv, dk), dtype=torch.float64, device=DEV) if s["S0"] is None else s["S0"].double()
    o, kept = torch.zeros_like(v), []
    for t in range(n):
        if back:
            kept.append(S)
        S, _ = _token(g[:, t, :, None, None] * S, k[:, t], v[:, t], beta[:, t])
        if not back:
            o[:, t] = torch.matmul(S, q[:, t, :, :, None])[..., 0]
    if not back:
        return dict(o=packed(o, s["o"]), S_out=S)
    do = padded(s["d_o"])
    dq, dkk, dvv, dbeta, dlog_g = (torch.zeros_like(x) for x in (q, k, v, beta, g))
    dS = torch.zeros_like(S) if s["dS_out"] is None else s["dS_out"].double()
    for t in reversed(range(n)):
        p = g[:, t, :, None, None] * kept.pop()
        S, w = _token(p, k[:, t], v[:, t], beta[:, t])
        dq[:, t] = torch.matmul(S.mT, do[:, t, :, :, None])[..., 0]
        dS = dS + do[:, t, :, :, None] * q[:, t, :, None, :]
        along = torch.matmul(dS, k[:, t, :, :, None])[..., 0]
        dbeta[:, t] = (along * w).sum(-1)
        dw = beta[:, t, :, None] * along
        dvv[:, t] = dw
        dkk[:, t] = beta[:, t, :, None] * torch.matmul(dS.mT, w[..., None])[..., 0] - torch.matmul(p.mT, dw[..., None])[..., 0]
        dP = dS - dw[..., None] * k[:, t, :, None, :]
        dlog_g[:, t] = (p * dP).sum((-1, -2))
        dS = g[:, t, :, None, None] * dP
    heads = lambda x: x.unflatten(2, (case["hk"], share)).sum(3)  # noqa: E731
    return dict(dq=packed(heads(dq), s["dq"]), dk=packed(heads(dkk), s["dk"]), dv=packed(dvv, s["dv"]),
                dbeta=packed(dbeta, s["dbeta"]), dlog_g=packed(dlog_g, s["dlog_g"]),
                dS0=dS if case["prior"] else None)


def _exact_step(case, s):
    share = case["hv"] // case["hk"]
    state = s["state"].double()
    for i, slot in enumerate(s["slot"].tolist()):
        k = s["k"][i].double().repeat_interleave(share, 0)
        state[slot], _ = _token(s["g"][i].double()[:, None, None] * state[slot], k, s["v"][i].double(),
                                s["beta"][i].double())
    q = s["q"].double().repeat_interleave(share, 1)
    return dict(o=torch.matmul(state[s["slot"].long()], q[..., None])[..., 0], state=state)


def _exact_scores(case, s):
    """Row blocks, so that a block's 64-bit copies stay small."""
    size = max(1, 2 ** 26 // case["vocab"])
    parts = []
    for r in range(0, case["rows"], size):
        x = s["logits"][r:r + size].double()
        logp = torch.log_softmax(x, 1)
        p = logp.exp()
        token = s["tokens"][r:r + size].long()[:, None]
        if case["op"] == "scores":
            got = dict(logp=logp.gather(1, token)[:, 0], entropy=-torch.xlogy(p, p).sum(1), lse=torch.logsumexp(x, 1))
            if case["topk"]:
                order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["topk"]]
                got.update(top_logp=logp.gather(1, order), top_tok=order.to(torch.int32))
        else:
            # the gradient with regard to the log-probabilities, then through the softmax
            ge = s["d_entropy"][r:r + size].double()[:, None]
            d = torch.where(p > 0, -ge * (logp + 1) * p, 0.0)
            d.scatter_add_(1, token, s["d_logp"][r:r + size].double()[:, None])
            if case["topk"]:
                d.scatter_add_(1, s["top_tok"][r:r + size].long(), s["d_top_logp"][r:r + size].double())
            got = dict(d=d - p * d.sum(1, keepdim=True))
        parts.append(got)
    whole = {key: torch.cat([x[key] for x in parts]) for key in parts[0]}
    return whole["d"] if case["op"] == "scores_grad" else whole


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("forward", "backward"):
        return _exact_rule(case, s)
    return _exact_step(case, s) if case["op"] == "step" else _exact_scores(case, s)


# ---------------------------------------------------------------- work

def work(case):
    e = 4 if case["io"] == "f32" else 2
    if case["op"] in ("scores", "scores_grad"):
        n = case["rows"] * case["vocab"]
        small = case["rows"] * (16 + 8 * case["topk"])
        return {"bytes": n * e * (1 if case["op"] == "scores" else 2) + small, "flops": 6 * n}
    hk, hv, dk, dv = (case[x] for x in ("hk", "hv", "dk", "dv"))
    state = 4 * hv * dk * dv
    row = e * (2 * hk * dk + 2 * hv * dv) + 8 * hv
    if case["op"] == "step":
        return {"bytes": case["batch"] * (row + 2 * state), "flops": case["batch"] * hv * 6 * dk * dv}
    rows, b = int(_lengths(np.random.default_rng(0), case).sum()), case["batch"]
    if case["op"] == "forward":
        return {"bytes": rows * row + b * state * (1 + case["prior"]), "flops": rows * hv * 6 * dk * dv}
    return {"bytes": 2 * rows * row + b * state * 3 * case["prior"], "flops": rows * hv * 18 * dk * dv}
