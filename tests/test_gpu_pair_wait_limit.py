"""Waits that run out in the kernels of CTA pairs, without a fault: with the wait limit at one microsecond and contractions of
tens of microseconds per tile the roles of both CTAs give up at different places, let what they have in flight land and return.
The calls succeed, the status word reports it, and with the default limit back the same calls give the same results bit for
bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


# a long contraction in the first kernel of each pass, and in the second
@pytest.mark.parametrize("T,H,I", [(600, 16384, 264), (600, 264, 16384), (3000, 8192, 1032)])
@pytest.mark.parametrize("il", [0, 1])
def test_feed_forward(T, H, I, il, set_option):
    mb = _mb()
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    x, dout = rand(T, H).to(bf), rand(T, H).to(bf)
    W1, W2 = (rand(H, 2 * I) * H ** -0.5).to(bf), (rand(I, H) * I ** -0.5).to(bf)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    set_option("FFN_TILES", 2)

    def calls(h=None):
        seen = []
        f = mb.ffn_fwd(x, W1, W2, gate_up_layout=il, status=status)
        torch.cuda.synchronize()
        seen.append(int(status.item()))
        status.zero_()
        g = mb.ffn_bwd(dout, x, f["h"] if h is None else h, W1, W2, bias=True, gate_up_layout=il, status=status)
        torch.cuda.synchronize()
        seen.append(int(status.item()))
        status.zero_()
        return seen, [f["out"], f["h"]] + [g[k] for k in ("dx", "dW1", "dW2", "db1", "db2")]

    seen, first = calls()
    assert seen == [0, 0]
    set_option("WAIT_LIMIT_NS", 1000)
    for _ in range(3):
        assert calls(first[1])[0] == [mb.STATUS_TIMEOUT] * 2
    set_option("WAIT_LIMIT_NS", None)
    seen, again = calls(first[1])
    assert seen == [0, 0]
    assert all(torch.equal(a, b) for a, b in zip(first, again))
