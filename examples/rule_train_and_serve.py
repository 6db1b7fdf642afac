"""A small language model of one Gated DeltaNet layer, trained and served.

Training: ragged sequences through the rule and the scores of their next tokens, with the gradients of
both.  Serving: prompts of different lengths in one pass, then steps that draft a tree per prompt from
the scores' best alternatives, verify it, accept a path by the scores' best tokens, commit it, and take
the token after it by itself.  Tokens and states stay on the device.

    python examples/rule_train_and_serve.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tree_masked_gated_amd as T  # noqa: E402


def model(vocab=96, h_k=2, h_v=4, d=32, width=48, seed=0, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: (torch.randn(s, generator=gen) * s[0] ** -0.5).to(device)  # noqa: E731
    p = dict(embed=rnd(vocab, width) * vocab ** 0.5, q=rnd(width, h_k * d), k=rnd(width, h_k * d), v=rnd(width, h_v * d),
             beta=rnd(width, h_v), g=rnd(width, h_v), out=rnd(h_v * d, vocab))
    return p, (h_k, h_v, d, vocab)


def project(p, heads, tokens):
    """q, k, v, beta and ln g of rows of tokens; q and k of unit length, q scaled."""
    h_k, h_v, d, _ = heads
    x = p["embed"][tokens.long()]
    unit = lambda y: torch.nn.functional.normalize(y.unflatten(-1, (h_k, d)), dim=-1)  # noqa: E731
    return (unit(x @ p["q"]) * d ** -0.5, unit(x @ p["k"]), (x @ p["v"]).unflatten(-1, (h_v, d)),
            torch.sigmoid(x @ p["beta"]), torch.nn.functional.logsigmoid(x @ p["g"] + 3))


# ---------------------------------------------------------------- training


class Rule(torch.autograd.Function):
    """o of packed sequences; the gates come in as ln g, in whose terms the gradient is."""

    @staticmethod
    def forward(ctx, offsets, q, k, v, beta, log_g):
        d = T.rule_dims(offsets.numel() - 1, q.shape[1], v.shape[1], q.shape[2], v.shape[2], "f32")
        o, g = torch.empty_like(v), log_g.exp()
        T.gdn_rule_forward(d, offsets, q, k, v, beta, g, o, T.rule_workspace(d, q.shape[0]))
        ctx.save_for_backward(offsets, q, k, v, beta, g)
        ctx.d = d
        return o

    @staticmethod
    def backward(ctx, d_o):
        offsets, *x = ctx.saved_tensors
        grads = [torch.empty_like(y) for y in x]
        T.gdn_rule_backward(ctx.d, offsets, *x, d_o.contiguous(), *grads, T.rule_workspace(ctx.d, x[0].shape[0], True))
        return (None, *grads)


class Scores(torch.autograd.Function):
    """ln p of the given tokens, and the entropy, of rows of logits."""

    @staticmethod
    def forward(ctx, logits, tokens):
        d = T.score_dims(*logits.shape, 0, "f32")
        logp, entropy, lse = (torch.empty_like(logits[:, 0]) for _ in range(3))
        T.gdn_token_scores(d, logits, tokens, logp, entropy, lse, T.score_workspace(d))
        ctx.save_for_backward(logits, tokens, lse, entropy)
        ctx.d = d
        return logp, entropy

    @staticmethod
    def backward(ctx, d_logp, d_entropy):
        logits, tokens, lse, entropy = ctx.saved_tensors
        d_logits = torch.empty_like(logits)
        T.gdn_token_scores_backward(ctx.d, logits, tokens, lse, entropy, d_logp.contiguous(), d_entropy.contiguous(),
                                    d_logits)
        return d_logits, None


def loss_of(p, heads, tokens, offsets, rule, scores):
    """Mean -ln p of the next tokens less a part of the entropy.  The last row of a sequence has no next token."""
    o = rule(offsets, *(x.contiguous() for x in project(p, heads, tokens)))
    has_next = torch.ones(tokens.numel(), dtype=torch.bool, device=tokens.device)
    has_next[offsets[1:].long() - 1] = False
    rows = has_next.nonzero()[:, 0]
    logp, entropy = scores(o.flatten(1)[rows] @ p["out"], tokens[rows + 1])
    return -logp.mean() - 0.01 * entropy.mean()


def train(steps=4, sizes=(70, 9, 130), seed=0, on_step=None):
    p, heads = model(seed=seed)
    for w in p.values():
        w.requires_grad_(True)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    offsets = torch.tensor([0, *torch.tensor(sizes).cumsum(0)], dtype=torch.int32, device="cuda")
    step = torch.optim.SGD(p.values(), lr=0.1)
    for _ in range(steps):
        tokens = torch.randint(0, heads[3], (sum(sizes),), generator=gen, device="cuda").int()
        step.zero_grad()
        loss = loss_of(p, heads, tokens, offsets, Rule.apply, Scores.apply)
        loss.backward()
        if on_step is not None:
            on_step(dict(p=p, heads=heads, tokens=tokens, offsets=offsets, loss=loss))
        step.step()
    return p, heads


# ---------------------------------------------------------------- serving


def serve(p, heads, steps=4, sizes=(70, 1, 130), nodes=12, alternatives=4, seed=0, on_step=None):
    """Greedy tokens after prompts of these sizes.  `on_step(info)` sees each step's tensors."""
    h_k, h_v, d, vocab = heads
    p = {n: w.detach().bfloat16() for n, w in p.items()}
    gen = torch.Generator(device="cuda").manual_seed(seed)
    batch, n = len(sizes), sum(sizes)
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    empty = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731

    def rows(tokens):
        q, k, v, beta, log_g = (x.contiguous() for x in project(p, heads, tokens))
        return q, k, v, beta.float(), log_g.float().exp()

    def best(logits, count):
        """The best `count` tokens of every row, and their ln p."""
        dims = T.score_dims(*logits.shape, count, "bf16")
        logp, tok = torch.empty(len(logits), count, device="cuda"), zeros(len(logits), count)
        T.gdn_token_scores(dims, logits, None, None, None, None, T.score_workspace(dims), top_logp=logp, top_tok=tok)
        return logp, tok

    # the prompts
    rule, tree_dims = T.rule_dims(batch, h_k, h_v, d, d, "bf16"), T.dims(batch, nodes, h_k, h_v, d, d, "bf16")
    offsets = torch.tensor([0, *torch.tensor(sizes).cumsum(0)], dtype=torch.int32, device="cuda")
    prompt = torch.randint(0, vocab, (n,), generator=gen, device="cuda").int()
    o, state = empty(n, h_v, d), torch.zeros(batch, h_v, d, d, device="cuda")
    T.gdn_rule_forward(rule, offsets, *rows(prompt), o, T.rule_workspace(rule, n), S_out=state)
    last = o[offsets[1:].long() - 1]

    # the drafter: the model's own logits for the first token, a random head for each later node
    head = torch.randn(nodes * vocab, vocab, generator=gen, device="cuda").bfloat16()
    tree, build = T.TreeCache(tree_dims), T.build_dims(batch, nodes, alternatives, 4)
    parent, drafted, path = (zeros(batch, nodes) for _ in range(3))
    accepted, accept_len, token, path_len = (zeros(batch) for _ in range(4))
    o_tree = empty(batch, nodes, h_v, d)
    for _ in range(steps):
        logits = last.flatten(1) @ p["out"]
        draft_logits = torch.cat([logits, logits @ head.T], 1).view(batch * (nodes + 1), vocab)
        logp, tok = best(draft_logits, alternatives)
        T.gdn_tree_build(build, logp.view(batch, nodes + 1, -1), tok.view(batch, nodes + 1, -1), parent, drafted,
                         torch.empty(batch, nodes, device="cuda"))
        q, k, v, beta, g = rows(drafted)
        T.gdn_tree_verify(tree_dims, state, q, k, v, beta, g, parent, o_tree, tree)
        _, target = best(o_tree.view(batch * nodes, -1) @ p["out"], 1)
        _, root = best(logits, 1)
        T.gdn_tree_accept(tree_dims, parent, drafted, target.view(batch, nodes), root.view(batch), accepted, accept_len,
                          token)
        T.gdn_tree_commit(tree_dims, state, state, k, tree, accepted, path, path_len)
        # the token after the path
        last = empty(batch, h_v, d)
        T.gdn_rule_step(rule, *rows(token), state, last)
        if on_step is not None:
            on_step(dict(prompt=prompt, offsets=offsets, drafted=drafted, path=path, path_len=path_len, token=token,
                         state=state, rows=rows, last=last, target=target.view(batch, nodes), root=root.view(batch),
                         accepted=accepted, accept_len=accept_len))
    return state


if __name__ == "__main__":
    count = int(sys.argv[1]) if len(sys.argv) > 1 else 4
    trained = train(count, on_step=lambda s: print("loss %.4f" % s["loss"].item(), flush=True))
    serve(*trained, steps=count, on_step=lambda s: print("accepted", s["path_len"].tolist(), "then",
                                                         s["token"].tolist(), flush=True))
