"""The feed-forward oracle against finite differences and torch's float64 automatic differentiation."""
import numpy as np
import pytest
import torch

from oracle import ffn as of


def _inputs(T=5, H=6, I=4, seed=0):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(s) for s in ((T, H), (H, 2 * I), (I, H), (2 * I,), (H,), (T, H))]


@pytest.mark.parametrize("gelu", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_against_autograd_and_differences(gelu, interleaved):
    x, W1, W2, b1, b2, dout = _inputs()
    out, h = of.forward(x, W1, W2, b1, b2, gelu, interleaved)
    got = of.backward(dout, x, h, W1, W2, gelu, interleaved)
    t = {k: torch.tensor(v, requires_grad=True) for k, v in dict(x=x, W1=W1, W2=W2, b1=b1, b2=b2).items()}
    th = t["x"] @ t["W1"] + t["b1"]
    g, u = (th[:, 0::2], th[:, 1::2]) if interleaved else th.chunk(2, 1)
    act = torch.nn.functional.gelu if gelu else torch.nn.functional.silu
    tout = act(g) * u @ t["W2"] + t["b2"]
    assert np.allclose(out, tout.detach().numpy(), rtol=1e-12, atol=1e-12)
    (tout * torch.tensor(dout)).sum().backward()
    for n, k in (("dx", "x"), ("dW1", "W1"), ("dW2", "W2"), ("db1", "b1"), ("db2", "b2")):
        assert np.allclose(got[n], t[k].grad.numpy(), rtol=1e-11, atol=1e-11), n
    f = lambda xx: (of.forward(xx, W1, W2, b1, b2, gelu, interleaved)[0] * dout).sum()  # noqa: E731
    eps = 1e-6
    for i, j in ((0, 0), (2, 3), (4, 5)):
        d = np.zeros_like(x)
        d[i, j] = eps
        assert abs((f(x + d) - f(x - d)) / (2 * eps) - got["dx"][i, j]) < 1e-6


def test_split_and_join_are_inverse():
    h = np.arange(24.0).reshape(3, 8)
    for il in (False, True):
        assert np.array_equal(of.join(*of.split(h, il), il), h)
