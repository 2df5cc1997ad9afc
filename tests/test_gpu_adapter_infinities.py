"""Infinite inputs of the adapters: results are infinite, with their sign, or NaN where the formula in 64 bits is, and finite
elsewhere.  scale u and v enter their products as two bf16 numbers each; neither may meet an infinity as a zero or with the
other's opposite sign."""
import numpy as np
import pytest
import torch

from helpers import np64
from oracle import adapter as oa

pytestmark = pytest.mark.gpu


def _case(r, exact, what, T=70, H=64, N=72, n=3):
    import moe_expert_layer_routing_gb300 as mb
    gen = torch.Generator().manual_seed(r)
    if exact:   # small whole numbers and scales that are powers of two: sums that one bf16 number holds
        rand = lambda *s: torch.randint(0, 2, s, generator=gen) * 2.0 - 1.0  # noqa: E731
    else:
        rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = dict(x=rand(T, H), dy=rand(T, N), A=rand(n, r, H), B=rand(n, r, N), base=rand(T, N), dbase=rand(T, H))
    inf = float("inf")
    if what == "x":
        d["x"][5, 9], d["x"][40, 63], d["x"][41, 0] = inf, -inf, inf
    elif what == "dy":
        d["dy"][7, 71], d["dy"][30, 2], d["dy"][31, 2] = -inf, inf, inf
    else:
        d[what][0, 0, 3], d[what][1, r - 1, 60], d[what][2, r // 2, 0] = inf, -inf, inf
    d = {k: v.to(torch.bfloat16).cuda() for k, v in d.items()}
    d["scale"] = torch.tensor([0.5, 2.0, 1.0], device="cuda")
    d["ids"] = torch.randint(-1, n, (T, 1), generator=gen, dtype=torch.int32).cuda()
    d["meta"] = mb.route_meta(d["ids"], n, 128)
    return mb, d


def _same_kind(got, ref, name):
    got = np64(got)
    with np.errstate(all="ignore"):
        for kind in (np.isnan, np.isposinf, np.isneginf):
            assert np.array_equal(kind(got), kind(ref)), (name, kind.__name__)


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("r", [1, 5, 16, 33, 64, 100])
@pytest.mark.parametrize("what", ["x", "dy", "A", "B"])
def test_infinite_inputs(what, r, exact):
    mb, d = _case(r, exact, what)
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])
    torch.cuda.synchronize()
    ids = d["ids"].cpu().numpy()[:, 0]
    x, dy, A, B, scale, base, dbase, u = (np64(t) for t in (d["x"], d["dy"], d["A"], d["B"], d["scale"], d["base"], d["dbase"], f["u"]))
    with np.errstate(all="ignore"):
        y, u64 = oa.forward(x, A, B, ids, scale, base)
        dx, dA, dB = oa.backward(dy, x, u, A, B, ids, scale, dbase)
    for name, got, ref in (("u", f["u"], u64), ("y", f["y"], y), ("dx", g["dx"], dx), ("dA", g["dA"], dA), ("dB", g["dB"], dB)):
        _same_kind(got, ref, name)


def test_zero_sums_add_nothing():
    """A sum of zero enters as zeros: the row keeps its base bit for bit, a base of zeros stays zeros."""
    mb, d = _case(16, False, "x")
    d["x"].zero_()
    big = torch.full_like(d["B"], 3e38)
    f = mb.adapter_fwd(d["x"], d["A"], big, d["meta"], scale=d["scale"], base=d["base"])
    z = mb.adapter_fwd(d["x"], d["A"], big, d["meta"], scale=d["scale"])
    torch.cuda.synchronize()
    assert torch.equal(f["y"], d["base"]) and torch.all(z["y"] == 0)


def test_tiny_sums():
    """Sums around bf16's smallest number, 2^-133, are off by at most that much (and by 2^-16 of themselves) before the product."""
    mb, d = _case(8, True, "x")
    d["x"].zero_()
    d["x"][:, 0] = 1
    d["A"].zero_()
    d["A"][:, :, 0] = torch.tensor([2.0 ** -k for k in (112, 117, 120, 125, 127, 130, 132, 133)], device="cuda").bfloat16()
    d["B"].zero_()
    for k in range(8):
        d["B"][:, k, k] = 2.0 ** 100
    one = torch.ones(3, device="cuda")
    y = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=one)["y"]
    torch.cuda.synchronize()
    v = np64(d["A"][0, :, 0])
    have = d["ids"].cpu().numpy()[:, 0] >= 0
    ref = v * 2.0 ** 100
    bound = 2.0 ** 100 * (2.0 ** -133 + 2.0 ** -16 * v)
    bound = bound + 2.0 ** -8 * (ref + bound)       # y's own rounding
    assert np.all(np.abs(np64(y)[have][:, :8] - ref) <= bound) and np.all(np64(y)[:, 8:] == 0)
