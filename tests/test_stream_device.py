"""Calls without a stream go to the current device's, and so take no tensors of another one."""
import types

import pytest
import torch

T = pytest.importorskip("tree_masked_gated_amd")


def on(device):
    return types.SimpleNamespace(get_device=lambda: device)


@pytest.mark.parametrize("raw", [None, lambda device: {3: 77}[device]])
def test_tensors_of_another_device(monkeypatch, raw):
    monkeypatch.setattr(T, "_raw_stream", raw)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert T._stream(None, on(3)) == 77 and T._stream(5, on(2)) == 5
    with pytest.raises(ValueError, match="current device"):
        T._stream(None, on(2))


@pytest.mark.gpu
def test_calls_refuse_them(monkeypatch):
    """The calls as they are made, with another device said to be the current one."""
    x = torch.zeros(4, 1, 32, device="cuda")
    gate, off = torch.ones(4, 1, device="cuda"), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    d, rows = T.rule_dims(1, 1, 1, 32, 32, "f32"), [torch.empty_like(x) for _ in range(4)]
    step, state = T.rule_dims(4, 1, 1, 32, 32, "f32"), torch.zeros(4, 1, 32, 32, device="cuda")
    logits, v, s = torch.zeros(4, 10, device="cuda"), torch.zeros(4, device="cuda"), T.score_dims(4, 10, 0, "f32")
    grads = [torch.empty_like(gate) for _ in range(2)]
    ws, back, scores = T.rule_workspace(d, 4), T.rule_workspace(d, 4, True), T.score_workspace(s)
    calls = [lambda: T.gdn_rule_forward(d, off, x, x, x, gate, gate, rows[0], ws),
             lambda: T.gdn_rule_backward(d, off, x, x, x, gate, gate, x, *rows[1:], *grads, back),
             lambda: T.gdn_rule_step(step, x, x, x, gate, gate, state, rows[0]),
             lambda: T.gdn_token_scores(s, logits, None, None, v, None, scores),
             lambda: T.gdn_token_scores_backward(s, logits, None, v, None, None, None, torch.empty_like(logits))]
    for call in calls:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
