"""The binding's checks of the feed-forward block's and the adapters' tensors, on the CPU: the quick expression and the checks
that word the message refuse the same, and what the expression refuses is refused whatever those find."""
import pytest
import torch

import moe_expert_layer_routing_gb300 as mb

BF = torch.bfloat16


def _ffn(**k):
    d = dict(x=torch.zeros(4, 64, dtype=BF), W1=torch.zeros(64, 32, dtype=BF), W2=torch.zeros(16, 64, dtype=BF))
    d.update(k)
    return mb._ffn_args(d["x"], d["W1"], d["W2"], "ffn")


def _adapters(meta=None, **k):
    d = dict(x=torch.zeros(4, 64, dtype=BF), A=torch.zeros(2, 8, 64, dtype=BF), B=torch.zeros(2, 8, 72, dtype=BF))
    m = dict(expert_offsets=torch.zeros(3, dtype=torch.int32), x_gather_idx=torch.zeros(4, dtype=torch.int32),
             s_reverse_scatter_idx=torch.zeros(4, dtype=torch.int32))
    d.update(k)
    m.update(meta or {})
    return mb._adapter_args(d["x"], d["A"], d["B"], m, None, "adapter")


FFN = [dict(x=torch.zeros(4, 64)), dict(x=torch.zeros(4, 128, dtype=BF)[:, ::2]), dict(W1=torch.zeros(64, 32)),
       dict(W1=torch.zeros(72, 32, dtype=BF)), dict(W1=torch.zeros(32, 64, dtype=BF).t()), dict(W2=torch.zeros(16, 72, dtype=BF)),
       dict(W2=torch.zeros(16, 64)), dict(W2=torch.zeros(64, 16, dtype=BF).t())]
ADAPTERS = [dict(x=torch.zeros(4, 64)), dict(x=torch.zeros(4, 128, dtype=BF)[:, ::2]), dict(A=torch.zeros(2, 8, 72, dtype=BF)),
            dict(A=torch.zeros(2, 8, 64)), dict(A=torch.zeros(2, 64, 8, dtype=BF).transpose(1, 2)), dict(B=torch.zeros(2, 8, 72)),
            dict(B=torch.zeros(2, 72, 8, dtype=BF).transpose(1, 2)), dict(meta=dict(expert_offsets=torch.zeros(4, dtype=torch.int32))),
            dict(meta=dict(expert_offsets=torch.zeros(3))), dict(meta=dict(x_gather_idx=torch.zeros(5, dtype=torch.int32))),
            dict(meta=dict(x_gather_idx=torch.zeros(4, dtype=torch.int64))),
            dict(meta=dict(s_reverse_scatter_idx=torch.zeros(8, dtype=torch.int32)[::2]))]


@pytest.mark.parametrize("silent", [False, True])
@pytest.mark.parametrize("call,bad", [(_ffn, b) for b in FFN] + [(_adapters, b) for b in ADAPTERS])
def test_refused(call, bad, silent, monkeypatch):
    if silent:      # the wording checks let everything pass
        monkeypatch.setattr(mb, "_rows", lambda t, *a: t.stride(0))
        monkeypatch.setattr(mb, "_dense", lambda t, *a: None)
    with pytest.raises(mb.MoeError):
        call(**bad)


def test_taken():
    assert _ffn()[:3] == (4, 64, 16) and _adapters()[:5] == (4, 64, 72, 2, 8)
