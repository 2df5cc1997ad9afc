"""The layer norm, router, balance and 8-bit checkpoint kernels on tensors of more than 2^31 elements: the last rows,
whose offsets pass 32 bits, give the bits that the same rows give in a call of their own (other rows are zeros), and
the sums over all rows stay within (n + 64) 2^-24 of their magnitudes, n the rows that are not zero."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


def _rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("T,H", [((1 << 19) + 3, 4104), ((1 << 21) + 5, 1025)])
def test_layer_norm(T, H):
    mb = _mb()
    n = 70
    x, dy = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-n:] = _rand(n, H, seed=1)
    dy[-n:] = _rand(n, H, seed=2)
    gamma, beta = _rand(H, seed=3), _rand(H, seed=4)
    assert x.numel() > 1 << 31
    far, near = ((mb.layer_norm_fwd(r, gamma, beta), r, g) for r, g in ((x, dy), (x[-n:].clone(), dy[-n:].clone())))
    grads = [mb.layer_norm_bwd(g, r, gamma, out["mean"], out["rstd"]) for out, r, g in (far, near)]
    for k in ("y", "mean", "rstd"):
        assert torch.equal(far[0][k][-n:], near[0][k])
    assert torch.equal(far[0]["y"][0].float(), beta.bfloat16().float())      # a row of zeros
    assert torch.equal(grads[0]["dx"][-n:], grads[1]["dx"]) and not grads[0]["dx"][:5].any()
    xh = (near[1].double() - near[0]["mean"].double()[:, None]) * near[0]["rstd"].double()[:, None]
    for k, terms in (("dgamma", near[2].double() * xh), ("dbeta", near[2].double())):
        # (xh itself is rounded twice)
        assert ((grads[0][k].double() - terms.sum(0)).abs() <= (n + 64) * U * terms.abs().sum(0)).all()


def test_router_and_balance():
    mb = _mb()
    T, E, K, n = (1 << 24) + 3, 128, 8, 100
    alpha, beta = 0.5, 0.25
    logits = torch.zeros(T, E, device="cuda")
    logits[-n:] = 2 * _rand(n, E, seed=1)
    assert logits.numel() > 1 << 31
    out = mb.router_fwd(mb.ROUTER_TOPK_OVER_SOFTMAX, logits, K, alpha=alpha, beta=beta)
    own = mb.router_fwd(mb.ROUTER_TOPK_OVER_SOFTMAX, logits[-n:].clone(), K)
    for k in ("ids", "scores", "lse"):
        assert torch.equal(out[k][-n:], own[k])
    counts = torch.bincount(own["ids"].flatten(), minlength=E)
    counts[:K] += T - n                                                      # rows of zeros: the first K experts
    assert torch.equal(out["counts"].flatten().long(), counts)
    d = mb.balance_bwd(logits, out["lse"], out["counts"], K, alpha=alpha, beta=beta)
    d = d["dlogits"] if isinstance(d, dict) else d
    p = torch.softmax(logits[-n:].double(), 1)
    c = counts.double()
    lse = torch.logsumexp(logits[-n:].double(), 1, keepdim=True)
    bal = alpha * E / (K * float(T) * T) * p
    want = bal * (c - (p * c).sum(1, keepdim=True)) + 2 * beta / T * lse * p
    size = bal * (c + (p * c).sum(1, keepdim=True)) + 2 * beta / T * lse.abs() * p
    tol = (E + 64 + 8 * float(logits[-n:].abs().max())) * U
    assert ((d[-n:].double() - want).abs() <= 2 * tol * size).all()


def test_checkpoint():
    mb = _mb()
    E, I, B, n = 2, 2048, 1024, 200
    first, second = 150, 512 * 1024 + n          # expert 1: whole blocks, then n rows
    R = first + second
    h = torch.zeros(R, 2 * I, dtype=torch.bfloat16, device="cuda")
    h[-n:] = _rand(n, 2 * I, seed=1)
    assert h.numel() > 1 << 31
    ids = torch.ones(R, 1, dtype=torch.int32, device="cuda")
    ids[:first] = 0
    meta = mb.route_meta(ids, E, B)
    out = mb.glu_fwd(h, meta, B)
    back = mb.ckpt8_unpack(out["ckpt_q"], out["ckpt_sf"], meta, R)
    assert out["ckpt_q"].numel() > 1 << 31
    meta = mb.route_meta(ids[-n:], E, B)
    own = mb.glu_fwd(h[-n:].clone(), meta, B)
    own_back = mb.ckpt8_unpack(own["ckpt_q"], own["ckpt_sf"], meta, n)
    assert torch.equal(out["a"][-n:], own["a"]) and torch.equal(back[-n:], own_back)
    assert not out["a"][: first + 1024].any() and not back[: first + 1024].any()
