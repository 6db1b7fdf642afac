"""The example's decode steps: every operator of the attention layer in its place, checked against the
64-bit references step by step."""
import os
import sys

import numpy as np
import pytest
import torch

from attn_reference import ancestors, attend

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def rows_of(pool, table, slot, n, page):
    """The first n cached rows of a slot, [n][h_kv][d] in 64 bits."""
    ids = table[slot, :-(-n // page)].long()
    return pool[0, ids].reshape(-1, *pool.shape[3:])[:n].double().cpu().numpy()


def test_decode_steps():
    from attention_decode import decode
    seen, kept = [], {}

    def check(s):
        torch.cuda.synchronize()
        p, ctx, table = s["prompts"], s["ctx"].tolist(), s["table"]
        batch, nodes = s["parent"].shape
        page = s["kp"].shape[2]
        assert (s["status"] == 0).all()
        f64 = {x: s[x].double().cpu().numpy() for x in ("q", "k", "v", "o")}
        for b in range(batch):
            keys, values = (rows_of(s[x], table, p + b, ctx[b], page) for x in ("kp", "vp"))
            if b in kept:                        # what earlier steps appended is what is read now
                assert np.array_equal(kept[b][0], keys) and np.array_equal(kept[b][1], values)
            r = slice(b * nodes, (b + 1) * nodes)
            look = np.concatenate([np.ones((nodes, ctx[b]), dtype=bool),
                                   ancestors(s["parent"][b].tolist()) | np.eye(nodes, dtype=bool)], axis=1)
            group = f64["q"].shape[1] // keys.shape[1]
            for h in range(keys.shape[1]):
                want, tol = attend(f64["q"][r, h * group:(h + 1) * group], np.concatenate([keys[:, h], f64["k"][r, h]]),
                                   np.concatenate([values[:, h], f64["v"][r, h]]), look, keys.shape[-1] ** -0.5, "bf16")
                assert (np.abs(f64["o"][r, h * group:(h + 1) * group] - want) <= tol).all()
            n = int(s["path_len"][b])
            path = s["path"][b, :n].tolist()
            assert int(s["new_len"][b]) == ctx[b] + n
            kept[b] = [np.concatenate([old, f64[x][r][path]]) for x, old in (("k", keys), ("v", values))]
        seen.append(s["new_len"].tolist())

    end = decode(steps=5, on_step=check)
    torch.cuda.synchronize()
    assert len(seen) == 5 and seen[-1] != seen[0]
    # after the first prompt's answers are gone and the pool is compact, the others' rows are there
    p, held = end["prompts"], int((end["ref"] > 0).sum())
    assert int((end["ref"][:held] > 0).sum()) == held
    for b, (k, v) in kept.items():
        if b % p == 0:
            assert int(end["length"][p + b]) == 0 and int(end["held"][p + b]) == 0
            continue
        n = int(end["length"][p + b])
        assert n == len(k)
        assert np.array_equal(rows_of(end["kp"], end["table"], p + b, n, end["page"]), k)
        assert np.array_equal(rows_of(end["vp"], end["table"], p + b, n, end["page"]), v)
