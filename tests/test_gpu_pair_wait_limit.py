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


@pytest.mark.parametrize("bn", [256, 128])
@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("recompute", [False, True])
def test_expert_layer(precision, bn, recompute, set_option):
    from helpers import to_device
    from moe_expert_layer_routing_gb300 import inputs as mi
    mb = _mb()
    mx = precision == "mxfp8"
    cfg = mi.small_moe("pair_wait", T=8192, H=4096 if recompute else 1024, I=256, E=2, K=1, B=128, seed=62,
                       precision=mi.PREC_MXFP8 if mx else mi.PREC_BF16, affinity=mi.AFFINITY_ON_I if mx else mi.AFFINITY_ON_H)
    ids = torch.zeros(8192, 1, dtype=torch.int32)
    ids[0, 0] = 1
    d = to_device(mi.with_ids(mi.make_moe_inputs(cfg), ids))
    kw = dict(x=d.x, dout=d.dout, s=d.s, ids=d.ids)
    weights = dict(W1=d.W1, W2=d.W2)
    if recompute:
        weights["W1t"] = d.W1.transpose(1, 2).contiguous()
    else:
        kw["ckpt"] = d.ckpt
    for name, w in weights.items():
        if mx:
            kw[name + "_q"], kw[name + "_sf"] = mb.quantize_weights(w, cfg.fp8_w)
        else:
            kw[name] = w
    set_option("PAIR_GEMMS", 2)
    set_option("PAIR_TILE_N", bn)

    def call():
        got = mb.moe_bwd(E=cfg.E, I=cfg.I, block_size=cfg.block_size, precision=cfg.precision, affinity=cfg.affinity,
                         fp8_act=cfg.fp8_act, fp8_w=cfg.fp8_w, **kw)
        torch.cuda.synchronize()
        return int(got["status"].item()), {k: got[k].clone() for k in ("dx", "dW1", "dW2", "ds")}

    seen, first = call()
    assert seen == 0
    set_option("WAIT_LIMIT_NS", 1000)
    for _ in range(3):
        assert call()[0] & mb.STATUS_TIMEOUT
    set_option("WAIT_LIMIT_NS", None)
    seen, again = call()
    assert seen == 0
    assert all(torch.equal(first[k], again[k]) for k in first)
