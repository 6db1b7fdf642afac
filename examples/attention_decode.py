"""Decode steps of a model whose layers alternate between Gated DeltaNet and softmax attention.

Every prompt is cached once and answered several times.  A step drafts a tree per answer,
verifies it through one layer of each kind, accepts a path and commits it: the recurrent state
takes the path's writes, the paged cache takes its keys and values.  All bookkeeping stays on
the device.  Projections and the drafter are stood in for by random rows.

    python examples/attention_decode.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tree_masked_gated_amd as T  # noqa: E402


def draft(gen, batch, n, width):
    """Parents of a tree whose levels hold `width` nodes, each below a random one of the level above."""
    at = torch.arange(n, device="cuda")
    pick = torch.randint(0, width, (batch, n), generator=gen, device="cuda")
    parent = torch.where(at >= width, (at // width - 1) * width + pick, -1)
    return parent.to(torch.int32).contiguous()


def decode(steps=4, prompts=3, answers=2, nodes=16, h_q=8, h_kv=2, d=64, page=16, prompt_rows=45, seed=0,
           on_step=None):
    """Runs the steps and returns the final page state.  `on_step(info)` sees each step's tensors."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s, dtype=torch.bfloat16: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = prompts * (1 + answers)
    width = (-(-(prompt_rows + steps * nodes) // page) + 4) // 4 * 4    # so that every slot's row begins on 16 bytes
    n_pages = slots * width
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731

    # the cache: slots 0 .. prompts - 1 hold the prompts
    pages = T.page_dims(n_pages, page, slots, width)
    kp, vp = randn(1, n_pages, page, h_kv, d), randn(1, n_pages, page, h_kv, d)
    cache = T.PagedCache(kp, vp)
    ref, held, length = zeros(n_pages), zeros(slots), zeros(slots)
    table = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    src, dst, count, status = zeros(slots), zeros(slots), zeros(1), zeros(slots)

    def reserve(need):
        T.gdn_pages_reserve(pages, need, ref, table, held, length, src, dst, count, status)
        T.gdn_pages_copy(cache, src, dst, count)

    need = zeros(slots)
    need[:prompts] = prompt_rows
    reserve(need)
    length[:prompts] = prompt_rows
    # each prompt's answers share its pages until they write to them
    batch = prompts * answers
    T.gdn_pages_fork(pages, ints([i % prompts for i in range(batch)]), ints(list(range(prompts, slots))), ref,
                     table, held, length, zeros(batch))

    attn = T.attn_dims(batch, nodes, h_q, h_kv, d, "bf16")
    gdn = T.dims(batch, nodes, h_kv, h_kv, d, d, "bf16")
    rope = T.rope_dims(d, "half")
    freq = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    workspace = T.attn_workspace(attn)
    tree = T.TreeCache(gdn)
    state = randn(batch, h_kv, d, d, dtype=torch.float32) * 0.1
    rows = batch * nodes
    o, o_gdn = randn(rows, h_q, d), randn(batch, nodes, h_kv, d)
    accepted, accept_len, token, path_len, new_len = (zeros(batch) for _ in range(5))
    path = zeros(batch, nodes)
    room = zeros(slots)
    room[prompts:] = nodes
    for _ in range(steps):
        parent = draft(gen, batch, nodes, 4)
        # the recurrent layer: outputs of all nodes, and the tree's record
        gk = torch.nn.functional.normalize(randn(batch, nodes, h_kv, d).float(), dim=-1).bfloat16()
        beta, g = (torch.rand(batch, nodes, h_kv, generator=gen, device="cuda") for _ in range(2))
        T.gdn_tree_verify(gdn, state, gk, gk, randn(batch, nodes, h_kv, d), beta, g, parent, o_gdn, tree)
        # the attention layer: q, k and v are slices of one projection
        fused = randn(rows, h_q + 2 * h_kv, d)
        q, k, v = fused[:, :h_q], fused[:, h_q:h_q + h_kv], fused[:, h_q + h_kv:]
        ctx = length[prompts:].clone()
        T.gdn_attn_rope(attn, rope, q, k, freq, ctx, tree.depth, q, k)
        T.gdn_attn_verify(attn, cache, table[prompts:], ctx, q, k, v, tree.anc_mask, tree.tree_status, o,
                          workspace)
        # tokens: the verifier agrees with a child or it does not
        drafted, target = (torch.randint(0, 3, (batch, nodes), generator=gen, device="cuda").int() for _ in range(2))
        root = torch.randint(0, 3, (batch,), generator=gen, device="cuda").int()
        T.gdn_tree_accept(gdn, parent, drafted, target, root, accepted, accept_len, token)
        # commit: room for the largest path, then both layers' rows
        reserve(room)
        T.gdn_tree_commit(gdn, state, state, gk, tree, accepted, path, path_len)
        T.gdn_attn_commit(attn, cache, table[prompts:], ctx, k, v, path, path_len, new_len)
        if on_step is not None:
            on_step(dict(q=q, k=k, v=v, o=o, ctx=ctx, parent=parent, path=path, path_len=path_len,
                         new_len=new_len, status=status, kp=kp, vp=vp, table=table, prompts=prompts))
        length[prompts:] = new_len
    # the answers of the first prompt are done; the rest moves together
    drop = zeros(slots)
    drop[prompts::prompts] = 1
    T.gdn_pages_free(pages, drop, ref, table, held, length)
    moves, target, remap = zeros(n_pages), zeros(n_pages), zeros(n_pages)
    T.gdn_pages_compact(pages, ref, table, held, moves, target, count, remap)
    T.gdn_pages_copy(cache, moves, target, count)
    return dict(ref=ref, table=table, held=held, length=length, kp=kp, vp=vp, page=page, prompts=prompts)


if __name__ == "__main__":
    end = decode(int(sys.argv[1]) if len(sys.argv) > 1 else 4, on_step=lambda s: print(
        "accepted", s["path_len"].tolist(), "rows", s["new_len"].tolist(), flush=True))
    print("pages held", int((end["ref"] > 0).sum()), "rows", end["length"].tolist())
