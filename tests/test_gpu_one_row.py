"""One row out of a wider matrix, as a token's part of a fused projection: its stride is never used, so any is taken, and the
results are those of the dense row."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


@pytest.mark.parametrize("wide", [66, 192, 4001])
def test_feed_forward(wide):
    mb = _mb()
    gen = torch.Generator(device="cuda").manual_seed(wide)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    x, dout = rand(1, wide), rand(1, wide + 2)
    W1, W2 = rand(64, 64), rand(32, 64)
    for tiles in (1, 2):
        with mb.option("FFN_TILES", tiles):
            got = mb.ffn_fwd(x[:, :64], W1, W2)
            ref = mb.ffn_fwd(x[:, :64].clone(), W1, W2)
        assert torch.equal(got["out"], ref["out"]) and torch.equal(got["h"], ref["h"])
    g = mb.ffn_bwd(dout[:, :64], x[:, :64], ref["h"], W1, W2, bias=True)
    r = mb.ffn_bwd(dout[:, :64].clone(), x[:, :64].clone(), ref["h"], W1, W2, bias=True)
    assert all(torch.equal(g[k], r[k]) for k in r)


@pytest.mark.parametrize("adapter", [-1, 1])
def test_adapters_in_place_on_a_part_of_a_fused_projection(adapter):
    mb = _mb()
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    H, N, n, r = 64, 72, 3, 5
    x, qkv, dx, A, B = rand(1, H + 2), rand(1, 3 * N), rand(1, H + 10), rand(n, r, H), rand(n, r, N)
    meta = mb.route_meta(torch.tensor([[adapter]], dtype=torch.int32, device="cuda"), n, 128)
    before = qkv.clone()
    ref = mb.adapter_fwd(x[:, :H].clone(), A, B, meta, base=qkv[:, :N].clone())
    got = mb.adapter_fwd(x[:, :H], A, B, meta, base=qkv[:, :N], out=qkv[:, :N])
    assert torch.equal(qkv[:, :N], ref["y"]) and torch.equal(qkv[:, N:], before[:, N:]) and torch.equal(got["u"], ref["u"])
    dy, old = qkv[:, N:2 * N], dx.clone()
    ref = mb.adapter_bwd(dy.clone(), x[:, :H].clone(), got["u"], A, B, meta, base=dx[:, :H].clone())
    back = mb.adapter_bwd(dy, x[:, :H], got["u"], A, B, meta, base=dx[:, :H], out=dx[:, :H])
    assert torch.equal(dx[:, :H], ref["dx"]) and torch.equal(dx[:, H:], old[:, H:])
    assert torch.equal(back["dA"], ref["dA"]) and torch.equal(back["dB"], ref["dB"])
