"""The adapter oracle against torch's float64 automatic differentiation and finite differences."""
import numpy as np
import torch

from oracle import adapter as oa


def test_against_autograd_and_differences():
    rng = np.random.default_rng(1)
    T, H, N, n, r = 9, 6, 5, 3, 2
    x, dy, base = (rng.standard_normal(s) for s in ((T, H), (T, N), (T, N)))
    A, B = rng.standard_normal((n, r, H)), rng.standard_normal((n, r, N))
    scale = rng.random(n) + 0.5
    ids = np.array([0, 2, -1, 0, 0, 2, -1, 2, 0])
    y, u = oa.forward(x, A, B, ids, scale, base)
    t = {k: torch.tensor(v, requires_grad=True) for k, v in dict(x=x, A=A, B=B).items()}
    have = torch.tensor(ids >= 0)
    i = torch.tensor(np.maximum(ids, 0))
    tu = torch.einsum("th,trh->tr", t["x"], t["A"][i]) * have[:, None]
    ty = torch.tensor(base) + torch.tensor(scale)[i][:, None] * torch.einsum("tr,trn->tn", tu, t["B"][i])
    assert np.allclose(y, ty.detach().numpy(), atol=1e-12) and np.allclose(u, tu.detach().numpy(), atol=1e-12)
    (ty * torch.tensor(dy)).sum().backward()
    dx, dA, dB = oa.backward(dy, x, u, A, B, ids, scale, np.zeros((T, H)))
    for got, k in ((dx, "x"), (dA, "A"), (dB, "B")):
        assert np.allclose(got, t[k].grad.numpy(), atol=1e-11), k
    assert np.all(dA[1] == 0) and np.all(dB[1] == 0) and np.all(dx[2] == 0)
    f = lambda a: (oa.forward(x, a, B, ids, scale, base)[0] * dy).sum()  # noqa: E731
    d = np.zeros_like(A)
    d[2, 1, 3] = 1e-6
    assert abs((f(A + d) - f(A - d)) / 2e-6 - dA[2, 1, 3]) < 1e-6
