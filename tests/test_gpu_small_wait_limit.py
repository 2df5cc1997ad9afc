"""Waits that run out in the feed-forward block's kernel for few tokens, without a fault.  Its waits are short (a k-block's copies
and products), so with the limit at one nanosecond only some run out: one call in ten does not report it where a contraction has a
million terms, and the test calls until one has.  The calls succeed, and with the default limit back they give the same results."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("il", [0, 1])
def test_few_tokens(il, set_option):
    import moe_expert_layer_routing_gb300 as mb
    T, H, I = 256, 64, 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, W1, W2 = rand(T, H), rand(H, 2 * I) * 0.125, rand(I, H) * 2.0 ** -10
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    set_option("FFN_TILES", 1)

    def call():
        status.zero_()
        out = mb.ffn_fwd(x, W1, W2, gate_up_layout=il, save=False, status=status)["out"]
        torch.cuda.synchronize()
        return out, int(status.item())

    first, seen = call()
    assert seen == 0
    set_option("WAIT_LIMIT_NS", 1)
    seen = [call()[1] for _ in range(40)]
    assert set(seen) <= {0, mb.STATUS_TIMEOUT} and mb.STATUS_TIMEOUT in seen
    set_option("WAIT_LIMIT_NS", None)
    again, seen = call()
    assert seen == 0 and torch.equal(first, again)
