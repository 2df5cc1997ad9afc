"""The dense branch of a block as a program runs it: norm, a projection with its requests' adapters, the gated feed-forward
block, dropout onto the residual stream, and the backward pass of all of it, against float64 automatic differentiation;
captured, on two streams at once, and on more than 2^31 elements.

Bound of the chain, relative Frobenius: a value that is stored in bf16 is off by at most 2^-8 of itself, and no path from an
input to a result has more than ten such roundings (norm, projection, scale u, its sum, gate and up, a, out, dropout, and as
many backward); the products are random matrices of norm about one, which enlarge an error and the value it sits on alike."""
import numpy as np
import pytest
import torch

from helpers import np64, rel_fro
from oracle import dropout as od
from oracle import ffn as of

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
CHAIN = 10 * HALF
P, SEED, OFFSET, EPS = 0.2, 77, 5, 1e-5


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


def _block(T=384, H=256, I=192, n=3, r=16):
    gen = torch.Generator().manual_seed(11)
    rand = lambda s, *shape: (s * torch.randn(*shape, generator=gen)).to(torch.bfloat16).cuda()  # noqa: E731
    ids = torch.randint(-1, n, (T, 1), generator=gen).int().cuda()
    return dict(x=rand(1, T, H), dout=rand(1, T, H), gamma=1 + rand(0.1, H), Wp=rand(H ** -0.5, H, H), A=rand(H ** -0.5, n, r, H),
                B=rand(r ** -0.5, n, r, H), scale=(0.5 + torch.rand(n, generator=gen)).cuda(), W1=rand(H ** -0.5, H, 2 * I),
                W2=rand(I ** -0.5, I, H), b1=rand(0.1, 2 * I), b2=rand(0.1, H), ids=ids, n=n)


def _step(d, stream=None):
    """One forward and backward pass; the results a program keeps."""
    mb = _mb()
    k = dict(stream=stream)
    meta = mb.route_meta(d["ids"], d["n"], 128, stream=stream)
    norm = mb.layer_norm_fwd(d["x"], d["gamma"], eps=EPS, kind=mb.NORM_RMS, **k)
    z = norm["y"] @ d["Wp"].t()
    ad = mb.adapter_fwd(norm["y"], d["A"], d["B"], meta, scale=d["scale"], base=z, out=z, **k)
    f = mb.ffn_fwd(z, d["W1"], d["W2"], d["b1"], d["b2"], glu=mb.GLU_GEGLU, **k)
    y = mb.dropout_fwd(f["out"], P, SEED, OFFSET, residual=d["x"], **k)
    db = mb.dropout_bwd(d["dout"], P, SEED, OFFSET, **k)
    g = mb.ffn_bwd(db, z, f["h"], d["W1"], d["W2"], bias=True, glu=mb.GLU_GEGLU, **k)
    lin = mb.linear_bwd(g["dx"], d["Wp"], norm["y"], precision=mb.PREC_BF16, **k)
    ag = mb.adapter_bwd(g["dx"], norm["y"], ad["u"], d["A"], d["B"], meta, scale=d["scale"], base=lin["dX"], out=lin["dX"], **k)
    ng = mb.layer_norm_bwd(ag["dx"], d["x"], d["gamma"], None, norm["rstd"], dres=d["dout"], kind=mb.NORM_RMS, **k)
    return dict(y=y, x=ng["dx"], gamma=ng["dgamma"], Wp=lin["dW"], A=ag["dA"], B=ag["dB"], W1=g["dW1"], W2=g["dW2"], b1=g["db1"],
                b2=g["db2"])


def test_step_against_automatic_differentiation():
    d = _block()
    got = _step(d)
    torch.cuda.synchronize()
    q = {k: d[k].double().requires_grad_() for k in ("x", "gamma", "Wp", "A", "B", "W1", "W2", "b1", "b2")}
    T, H = d["x"].shape
    norm = q["x"] * torch.rsqrt((q["x"] ** 2).mean(1, keepdim=True) + EPS) * q["gamma"]
    ids = d["ids"][:, 0].long()
    rows = []
    for t in range(T):
        a = int(ids[t])
        rows.append(norm[t] @ q["Wp"].t() + (0 if a < 0 else d["scale"][a].double() * ((q["A"][a] @ norm[t]) @ q["B"][a])))
    gate, up = (torch.stack(rows) @ q["W1"] + q["b1"]).chunk(2, 1)
    out = (torch.nn.functional.gelu(gate) * up) @ q["W2"] + q["b2"]
    keep = torch.from_numpy(od.keep(T, H, P, SEED, OFFSET)).cuda()
    y = q["x"] + torch.where(keep, out / (1 - P), torch.zeros_like(out))
    (y * d["dout"].double()).sum().backward()
    assert rel_fro(np64(got["y"]), np64(y)) <= CHAIN
    for k in q:
        assert rel_fro(np64(got[k]), np64(q[k].grad)) <= CHAIN, k


def test_captured_step():
    d = _block(T=128)
    _step(d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = _step(d)
    for _ in range(2):
        d["x"].mul_(-0.75)
        d["ids"].copy_(d["ids"].roll(5, 0))
        g.replay()
        torch.cuda.synchronize()
        now = _step(d)
        torch.cuda.synchronize()
        assert all(torch.equal(now[k], held[k]) for k in now)


def test_two_streams_at_once():
    """Steps of different sizes that share the SMs' shared memory and TMEM."""
    big, small = _block(), _block(T=128, H=128, I=64, n=40, r=100)
    ref = [_step(big), _step(small)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for s, d in zip(streams, (big, small)):
            with torch.cuda.stream(s):
                got.append(_step(d))
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert all(torch.equal(out[k], ref[i % 2][k]) for k in out), i


def test_feed_forward_past_32_bits():
    """More than 2^31 pre-activations: the last rows' results against float64, dW over rows of which only they are not zero."""
    mb = _mb()
    T, H, I, tail = 270000, 64, 4096, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda s, *shape: s * torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x, dout = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), rand(1, T, H)
    dout[:-tail] = 0
    x[-tail:] = rand(1, tail, H)
    W1, W2 = rand(H ** -0.5, H, 2 * I), rand(I ** -0.5, I, H)
    f = mb.ffn_fwd(x, W1, W2)
    g = mb.ffn_bwd(dout, x, f["h"], W1, W2)
    torch.cuda.synchronize()
    w1, w2, xt, dt = np64(W1), np64(W2), np64(x[-tail:]), np64(dout[-tail:])
    out, h = of.forward(xt, w1, w2)
    assert rel_fro(np64(f["h"][-tail:]), h) <= HALF and rel_fro(np64(f["out"][-tail:]), out) <= 3 * HALF
    ref = of.backward(dt, xt, np64(f["h"][-tail:]), w1, w2)
    for k in ("dx", "dW1", "dW2"):
        assert rel_fro(np64(g[k][-tail:] if k == "dx" else g[k]), ref[k]) <= 3 * HALF, k
    assert torch.all(g["dx"][:-tail][-100:] == 0) and np.all(np64(f["out"][:100]) == 0)
