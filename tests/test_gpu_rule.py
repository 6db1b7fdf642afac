"""The gated delta rule over whole sequences on the GPU, against the token-by-token rule in 64 bits.

Tolerances (2-norm, per tensor).  fp32 results: a value passes through at most six sums (two
products with the state, the chunk's solve, the write, the read, the decay) of up to 256 products;
rounding errors of 2^-24 add at random, sqrt(256) 2^-24 = 1e-6 each, 6e-6 for six.  bf16 results:
one rounding of half a step, 2^-8, plus, for o, one of Y (2^-8) and two-term factors (2^-16); for
dq and dv none; for dk, two factors of 2^-8 each.

dS0 is measured against its terms too: it is the sum over the rows of a_t (q_t do_t^T - beta_t k_t
dR_t^T), a_t <= 1 the gates' product alone, and what later writes erase cancels only in the sum.  So
its error is 2^-24 of terms of the size |q_t| |do_t| each, which add at random, however small
the sum (with d_k = 1, 67 terms near 1 sum to 0.01: 67^(1/2) 2^-24 / 0.01 = 5e-5 of it).
"""
import pytest
import torch

import rule_reference as R

T = pytest.importorskip("tree_masked_gated_amd")
pytestmark = pytest.mark.gpu

F32 = 6e-6
HALF = 2.0 ** -8


def bound(name, io):
    if io == "f32" or name in ("S_out", "dbeta", "dlog_g", "dS0"):
        return F32
    return {"o": 2 * HALF, "dk": 3 * HALF}.get(name, HALF) + F32


def make(sizes, hk, hv, dk, dv, io, seed=0, prior=True, gates="mixed", fused=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    n, dt = sum(sizes), torch.float32 if io == "f32" else torch.bfloat16
    x = dict(q=rnd(n, hk, dk) * dk ** -0.5, k=torch.nn.functional.normalize(rnd(n, hk, dk), dim=-1), v=rnd(n, hv, dv),
             d_o=rnd(n, hv, dv))
    x = {a: b.to(dt) for a, b in x.items()}
    if fused:                                        # slices of one projection's output, heads of unequal strides
        wide = torch.cat([x["q"], x["k"], x["v"]], 1)
        x.update(q=wide[:, :hk], k=wide[:, hk:2 * hk], v=wide[:, 2 * hk:])
    x["beta"] = torch.rand(n, hv, generator=gen, device="cuda")
    rate = {"mixed": torch.logspace(-3, 0, hv, device="cuda"), "none": torch.zeros(hv, device="cuda"),
            "strong": torch.full((hv,), 20.0, device="cuda")}[gates]
    x["g"] = torch.exp(-rate * torch.rand(n, hv, generator=gen, device="cuda"))
    off = [0]
    for s in sizes:
        off.append(off[-1] + s)
    x["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    b = len(sizes)
    x["S0"] = 0.3 * rnd(b, hv, dv, dk) if prior else None
    x["dS_out"] = 0.3 * rnd(b, hv, dv, dk) if prior else None
    x["dims"] = T.rule_dims(b, hk, hv, dk, dv, io)
    return x


ARGS = ("q", "k", "v", "beta", "g")


def forward(x, stream=None, ws=None, **out):
    o = out.get("o", torch.empty(x["v"].shape, dtype=x["v"].dtype, device="cuda"))
    d = x["dims"]
    S = out.get("S_out", torch.empty(d.batch, d.h_v, d.d_v, d.d_k, device="cuda"))
    ws = T.rule_workspace(d, x["q"].shape[0]) if ws is None else ws
    T.gdn_rule_forward(d, x["offsets"], *(x[a] for a in ARGS), o, ws, S0=x["S0"], S_out=S, stream=stream)
    return dict(o=o, S_out=S)


def grads_like(x):
    e = lambda a: torch.empty(x[a].shape, dtype=x[a].dtype, device="cuda")  # noqa: E731
    d = x["dims"]
    return dict(dq=e("q"), dk=e("k"), dv=e("v"), dbeta=e("beta"), dlog_g=e("g"),
                dS0=torch.empty(d.batch, d.h_v, d.d_v, d.d_k, device="cuda"))


def backward(x, stream=None, ws=None, out=None):
    out = grads_like(x) if out is None else out
    ws = T.rule_workspace(x["dims"], x["q"].shape[0], backward=True) if ws is None else ws
    T.gdn_rule_backward(x["dims"], x["offsets"], *(x[a] for a in ARGS), x["d_o"],
                        *(out[a] for a in ("dq", "dk", "dv", "dbeta", "dlog_g")), ws, S0=x["S0"], dS_out=x["dS_out"],
                        dS0=out["dS0"], stream=stream)
    return out


def reference(x):
    return R.batch(x["offsets"].tolist(), *(x[a] for a in ARGS), x["S0"], x["d_o"], x["dS_out"])


def check(x, got, io):
    want = reference(x)
    for name, value in got.items():
        most = bound(name, io)
        if name == "dS0":
            share = x["v"].shape[1] // x["q"].shape[1]
            terms = x["q"].double().norm(dim=-1).repeat_interleave(share, 1) * x["d_o"].double().norm(dim=-1)
            most *= 1 + terms.norm().item() / want[name].norm().item()
        assert R.rel(value, want[name]) <= most, (name, R.rel(value, want[name]))


CASES = [
    # sizes, hk, hv, dk, dv: lengths around the chunk of 64 rows, empty ones, shared heads, odd head sizes
    ([1], 1, 1, 128, 128), ([64], 1, 2, 128, 128), ([65, 0, 63, 1], 2, 4, 128, 128), ([0, 130, 0], 1, 4, 64, 64),
    ([200, 17], 2, 2, 128, 64), ([33, 128], 1, 3, 48, 80), ([70, 5], 2, 2, 256, 256), ([90], 1, 2, 96, 33),
    ([67], 1, 1, 1, 1), ([66], 2, 2, 200, 17), ([300], 1, 2, 16, 130),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,hk,hv,dk,dv", CASES)
def test_forward_and_backward(sizes, hk, hv, dk, dv, io):
    x = make(sizes, hk, hv, dk, dv, io)
    check(x, {**forward(x), **backward(x)}, io)


# Batches of many sequences, most of them empty or short, for which the scans take wider slices; with no more
# than 64 sequences the longest go first.
MANY = [(60, 4, 8, 64, 80), (70, 2, 4, 128, 128), (60, 4, 12, 100, 33), (20, 4, 8, 128, 128), (36, 2, 4, 48, 128),
        (20, 2, 4, 200, 96)]


def many(batch, *heads, io):
    sizes = [3, 0, 130, 1, 64, 65, 0, 200, 63, 2] + [i % 3 for i in range(batch - 10)]
    return make(sizes, *heads, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("batch,hk,hv,dk,dv", MANY)
def test_many_sequences(batch, hk, hv, dk, dv, io):
    x = many(batch, hk, hv, dk, dv, io=io)
    check(x, {**forward(x), **backward(x)}, io)


@pytest.mark.parametrize("skip", [0, 1])
def test_many_sequences_in_slices_of_one_projection(skip):
    """Rows that are whole operands as they lie, and the same ones an element further, which are not."""
    x = many(70, 2, 4, 128, 128, io="bf16")
    want = forward(x)
    wide = torch.cat([x["q"][:, :0].new_zeros(x["q"].shape[0], 1, 128)] + [x[a] for a in ("q", "k", "v")], 1).flatten(1)
    wide = torch.nn.functional.pad(wide, (0, 8)).roll(skip, 1)
    at = lambda h, n: wide[:, (1 + h) * 128 + skip:(1 + h + n) * 128 + skip].unflatten(1, (n, 128))  # noqa: E731
    y = {**x, "q": at(0, 2), "k": at(2, 2), "v": at(4, 4)}
    assert all(torch.equal(x[a], y[a]) for a in ("q", "k", "v"))
    got = forward(y)
    assert all(torch.equal(got[a], want[a]) for a in want)


@pytest.mark.parametrize("batch,dv", [(2, 128), (20, 128), (70, 128), (70, 33)])
def test_outputs_in_a_wider_tensor(batch, dv):
    """Outputs at odd places between others, which stay as they were."""
    x = many(batch, 2, 4, 128, dv, io="bf16") if batch > 9 else make([67, 130], 2, 4, 128, dv, "bf16")
    want, n = forward(x)["o"], x["v"].shape[0]
    wide = torch.full((n, 4, dv + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    for at in (1, 4, 8):
        wide.fill_(7)
        forward(x, o=wide[:, :, at:at + dv])
        assert torch.equal(wide[:, :, at:at + dv], want)
        assert (wide[:, :, :at] == 7).all() and (wide[:, :, at + dv:] == 7).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_without_states(io):
    """No state before, none asked for; dS_out and dS0 neither."""
    x = make([70, 3], 1, 2, 64, 64, io, prior=False)
    o, out = torch.empty_like(x["v"]), grads_like(x)
    T.gdn_rule_forward(x["dims"], x["offsets"], *(x[a] for a in ARGS), o, T.rule_workspace(x["dims"], 73))
    T.gdn_rule_backward(x["dims"], x["offsets"], *(x[a] for a in ARGS), x["d_o"],
                        *(out[a] for a in ("dq", "dk", "dv", "dbeta", "dlog_g")),
                        T.rule_workspace(x["dims"], 73, backward=True))
    del out["dS0"]
    check(x, dict(o=o, **out), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (40, 40), (33, 33)])
def test_slices_of_one_projection(dk, dv, io):
    """Inputs and outputs with strides, aligned and not."""
    x = make([100, 30], 2, 4, dk, dv, io, fused=True)
    wide = torch.empty(130, 8, dk, dtype=x["v"].dtype, device="cuda")
    out = {**grads_like(x), "dq": wide[:, :2], "dk": wide[:, 2:4], "dv": wide[:, 4:]}
    heads_first = torch.empty(4, 130, dv, dtype=x["v"].dtype, device="cuda")
    check(x, {**forward(x, o=heads_first.transpose(0, 1)), **backward(x, out=out)}, io)


@pytest.mark.parametrize("gates", ["none", "strong"])
def test_gates(gates):
    """Gates of 1 throughout, and gates whose running product leaves the range of fp32 within a chunk."""
    x = make([150], 1, 2, 64, 64, "f32", gates=gates)
    x["g"][3] = 1e-38
    check(x, {**forward(x), **backward(x)}, "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gates_of_zero(io):
    """A gate of 0 forgets everything before its row, and its gradient with regard to ln g is 0."""
    x = make([70, 130, 1], 2, 4, 64, 64, io)
    zero = torch.rand(x["g"].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(8)) < 0.1
    zero[[0, 64, 70, 199], :2] = True
    x["g"][zero] = 0
    got = {**forward(x), **backward(x)}
    check(x, got, io)
    assert (got["dlog_g"][zero] == 0).all()


def test_write_strengths():
    """No writes at all, whole writes, and the same key every time."""
    x = make([100, 80], 1, 2, 64, 64, "f32", gates="none")
    x["beta"][:50] = 0
    x["beta"][50:100] = 1
    x["k"][100:] = x["k"][100]
    x["beta"][100:] = 0.9
    check(x, {**forward(x), **backward(x)}, "f32")


def test_gradients_are_those_of_differences():
    """The calls against each other: central differences of the forward call along random directions, in fp32
    with steps large enough to be seen: the value's rounding, 2^-24 of sums of n terms, over the step, and the
    step squared times a third derivative of the value's size."""
    x = make([90], 1, 2, 32, 32, "f32")
    gen = torch.Generator(device="cuda").manual_seed(5)

    def value(**kw):
        y = forward({**x, **kw})
        return (y["o"].double() * x["d_o"].double()).sum() + (y["S_out"].double() * x["dS_out"].double()).sum()
    got = backward(x)
    scale = sum((x[a].double() * got[b].double()).norm() for a, b in (("q", "dq"), ("v", "dv")))
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("beta", "dbeta"), ("g", "dlog_g"), ("S0", "dS0")):
        along = torch.randn(x[name].shape, generator=gen, device="cuda")
        along *= 1 / along.norm()
        h = 2e-2
        move = (lambda e: x["g"] * torch.exp(e * along)) if name == "g" else (lambda e: x[name] + e * along)  # noqa
        diff = (value(**{name: move(h)}) - value(**{name: move(-h)})) / (2 * h)
        want = (got[key].double() * along).sum()
        assert abs(diff - want) <= 1e-3 * max(abs(want), scale, got[key].norm()), name


def test_rows_behind_the_last_sequence_and_unusable_sequences():
    x = make([40, 70, 20], 1, 2, 64, 64, "f32")
    good = {**forward(x), **backward(x)}
    n = 130
    y = dict(x)
    # rows 110 .. 129 belong to nobody now; sequence 2's offsets pass the rows
    y["offsets"] = torch.tensor([0, 40, 110, 200], dtype=torch.int32, device="cuda")
    keep = {k: torch.full_like(v, 7.0) for k, v in good.items()}
    got = {**forward(y, o=keep["o"], S_out=keep["S_out"]), **backward(y, out=keep)}
    for name, value in got.items():
        if value.shape[0] == n:
            assert torch.equal(value[:110], good[name][:110]), name
            assert (value[110:] == 7).all(), name
        else:
            assert torch.equal(value[:2], good[name][:2]), name
    assert torch.equal(got["S_out"][2], x["S0"][2]) and torch.equal(got["dS0"][2], x["dS_out"][2])
    for off in ([-1, 40, 110, 130], [0, 40, 30, 130]):
        y["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        got = forward(y)
        bad = 0 if off[0] < 0 else 1
        assert torch.equal(got["S_out"][bad], x["S0"][bad])


def test_no_rows_and_no_sequences():
    x = make([0, 0], 1, 2, 64, 64, "bf16")
    got = {**forward(x), **backward(x)}
    assert torch.equal(got["S_out"], x["S0"]) and torch.equal(got["dS0"], x["dS_out"])
    x = make([], 1, 2, 64, 64, "bf16")
    x["offsets"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    forward(x)
    backward(x)
    torch.cuda.synchronize()


def test_state_in_place_and_pieces():
    """A prompt in pieces, each from the state that the last one left in place, is the prompt at once."""
    x = make([300], 2, 4, 128, 128, "f32")
    whole = forward(x)
    S, outs, at = x["S0"].clone(), [], 0
    for n in (1, 100, 64, 135):
        y = {**x, **{a: x[a][at:at + n] for a in ARGS}, "S0": S}
        y["offsets"] = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        outs.append(forward(y, S_out=S)["o"])
        at += n
    assert R.rel(torch.cat(outs), whole["o"]) <= 2 * F32 and R.rel(S, whole["S_out"]) <= 2 * F32
    back = backward(x)
    d = x["dS_out"].clone()
    out = {**grads_like(x), "dS0": d}
    backward({**x, "dS_out": d}, out=out)
    assert torch.equal(d, back["dS0"])


def test_runs_alike_streams_and_shared_workspace():
    """The same bits from run to run, on a stream of its own, with a workspace that a larger call has used, and
    from a captured graph that is replayed among eager calls with it."""
    x, big = make([130, 20], 1, 4, 128, 128, "bf16"), make([400, 90], 2, 4, 128, 128, "bf16", seed=3)
    first = {**forward(x), **backward(x)}
    ws = T.rule_workspace(big["dims"], 490, backward=True)
    ws.fill_(255)                                    # NaN patterns in every place
    forward(big, ws=ws)
    backward(big, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = {**forward(x, ws=ws), **backward(x, ws=ws)}
    side.synchronize()
    for name in first:
        assert torch.equal(first[name], again[name]), name
    out, f = grads_like(x), dict(o=torch.empty_like(x["v"]), S_out=torch.empty_like(x["S0"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(x, ws=ws, **f)
        backward(x, ws=ws, out=out)
    for _ in range(3):
        for v in (*out.values(), *f.values()):
            v.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for name, v in {**out, **f}.items():
            assert torch.equal(first[name], v), name
        backward(big, ws=ws)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("batch,hk,hv,dk,dv", [(1, 1, 1, 128, 128), (5, 2, 4, 64, 64), (3, 1, 2, 256, 256),
                                               (4, 2, 2, 48, 80), (2, 1, 3, 33, 130), (2, 1, 1, 1, 1),
                                               (7, 1, 2, 128, 40)])
def test_step(batch, hk, hv, dk, dv, io):
    """Tokens one at a time are the sequence: outputs and states, on slots of a pool in any order; and a state
    that no sequence has stays."""
    steps, slots = 3, batch + 2
    x = make([steps] * batch, hk, hv, dk, dv, io, fused=dk == dv)
    slot = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:batch].to(torch.int32).cuda()
    pool = torch.full((slots, hv, dv, dk), 5.0, device="cuda")
    pool[slot.long()] = x["S0"]
    outs = []
    for t in range(steps):
        at = torch.arange(batch, device="cuda") * steps + t
        o = torch.empty(batch, hv, dv, dtype=x["v"].dtype, device="cuda")
        T.gdn_rule_step(x["dims"], *(x[a][at] for a in ARGS), pool, o, slot=slot)
        outs.append(o)
    want = reference(x)
    o = torch.stack(outs, 1).flatten(0, 1)
    assert R.rel(o, want["o"]) <= (F32 if io == "f32" else HALF + F32)
    assert R.rel(pool[slot.long()], want["S_out"]) <= F32
    free = [s for s in range(slots) if s not in slot.tolist()]
    assert (pool[free] == 5).all()


def test_step_slots():
    """Absent tokens, slots outside the pool, and a slot that two sequences name."""
    x = make([1] * 6, 1, 2, 64, 64, "f32")
    pool = x["S0"][:4].clone()
    before, o = pool.clone(), torch.full((6, 2, 64), 9.0, device="cuda")
    slot = torch.tensor([2, -1, 4, 2, -7, 0], dtype=torch.int32, device="cuda")
    args = [x[a] for a in ARGS]
    T.gdn_rule_step(x["dims"], *args, pool, o, slot=slot)
    alone, single = before.clone(), torch.empty_like(o)
    T.gdn_rule_step(x["dims"], *args, alone, single, slot=torch.tensor([2, -1, -1, -1, -1, 0], dtype=torch.int32,
                                                                     device="cuda"))
    assert torch.equal(pool, alone) and torch.equal(pool[[1, 3]], before[[1, 3]])
    assert torch.equal(o[[0, 5]], single[[0, 5]]) and (o[1] == 9).all() and o[[2, 3, 4]].isnan().all()
    whole = x["S0"].clone()                          # without slots: sequence b's is b
    T.gdn_rule_step(x["dims"], *args, whole, o)
    order = x["S0"].clone()
    T.gdn_rule_step(x["dims"], *args, order, single, slot=torch.arange(6, dtype=torch.int32, device="cuda"))
    assert torch.equal(whole, order) and torch.equal(o, single)


def test_step_follows_forward():
    """A prompt, then tokens: the states and outputs of the longer prompt."""
    x = make([70, 70], 1, 2, 128, 128, "f32")
    head, at = {a: torch.cat([x[a][:66], x[a][70:136]]) for a in ARGS}, torch.tensor([66, 136], device="cuda")
    y = {**x, **head, "offsets": torch.tensor([0, 66, 132], dtype=torch.int32, device="cuda")}
    S, whole = forward(y)["S_out"], forward(x)
    for t in range(4):
        o = torch.empty(2, 2, 128, device="cuda")
        T.gdn_rule_step(x["dims"], *(x[a][at + t] for a in ARGS), S, o)
        assert R.rel(o, whole["o"][at + t]) <= 2 * F32
    assert R.rel(S, whole["S_out"]) <= 2 * F32


def test_agrees_with_the_tree_call():
    """A chain is a sequence: gdn_tree_verify and gdn_tree_commit of a chain of 100 nodes."""
    x = make([100, 100], 2, 4, 128, 128, "bf16")
    d = T.dims(2, 100, 2, 4, 128, 128, "bf16")
    cache, o = T.TreeCache(d), torch.empty(2, 100, 4, 128, dtype=torch.bfloat16, device="cuda")
    par = torch.arange(-1, 99, dtype=torch.int32, device="cuda").repeat(2, 1)
    t = {a: x[a].reshape(2, 100, *x[a].shape[1:]) for a in ARGS}
    T.gdn_tree_verify(d, x["S0"], t["q"], t["k"], t["v"], t["beta"], t["g"], par, o, cache)
    S, path = torch.empty_like(x["S0"]), torch.empty(2, 100, dtype=torch.int32, device="cuda")
    last, n = torch.full((2,), 99, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    T.gdn_tree_commit(d, x["S0"], S, t["k"], cache, last, path, n)
    got = forward(x)
    # the tree kernels' own bound is 1e-2
    assert R.rel(got["o"], o.flatten(0, 1)) <= 1e-2 + bound("o", "bf16") and R.rel(got["S_out"], S) <= 1e-2 + F32


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_many_sequences_run_alike(io):
    """The wider scans: the same bits with NaN patterns in the workspace, beside another call on another stream, and
    from replays of a captured graph."""
    x, other = many(70, 2, 4, 128, 128, io=io), make([200, 65], 2, 4, 128, 128, io, seed=5)
    first, alone = {**forward(x), **backward(x)}, {**forward(other), **backward(other)}
    ws = T.rule_workspace(x["dims"], x["q"].shape[0], backward=True)
    ws.fill_(255)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        beside = {**forward(other), **backward(other)}
    again = {**forward(x, ws=ws), **backward(x, ws=ws)}
    torch.cuda.synchronize()
    for name in first:
        assert torch.equal(first[name], again[name]) and torch.equal(alone[name], beside[name]), name
    out, f = grads_like(x), dict(o=torch.empty_like(x["v"]), S_out=torch.empty_like(x["S0"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(x, ws=ws, **f)
        backward(x, ws=ws, out=out)
    for _ in range(3):
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for name, v in {**out, **f}.items():
            assert torch.equal(first[name], v), name
        forward(other)
