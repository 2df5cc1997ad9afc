"""Pins of the oracles oracle/norm.py, oracle/balance.py and oracle/ckpt8.py: finite differences, torch's own
float64 operators, closed forms and hand-worked groups."""
import numpy as np
import pytest
import torch

from oracle import balance as ob
from oracle import ckpt8 as oc
from oracle import norm as on


def _fd(f, v, h=1e-6):
    g = np.zeros_like(v)
    for i in np.ndindex(*v.shape):
        a, b = v.copy(), v.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("kind", [on.LAYER, on.RMS])
@pytest.mark.parametrize("H", [1, 2, 13])
def test_norm_backward_by_differences(kind, H):
    rng = np.random.default_rng(H)
    x, dy, dres = (rng.standard_normal((3, H)) for _ in range(3))
    gamma, beta = rng.standard_normal(H), rng.standard_normal(H)
    loss = lambda x, g, b: np.sum(dy * on.forward(x, g, b, 1e-2, kind)[0]) + np.sum(dres * x)  # noqa: E731
    dx, dg, db = on.backward(dy, x, gamma, 1e-2, kind, dres)
    for got, num in ((dx, _fd(lambda v: loss(v, gamma, beta), x)), (dg, _fd(lambda v: loss(x, v, beta), gamma)),
                     (db, _fd(lambda v: loss(x, gamma, v), beta))):
        # central differences with h = 1e-6: rounding 1e-16 |loss| / h ~ 1e-9, truncation ~ h^2
        np.testing.assert_allclose(got, num, rtol=1e-6, atol=1e-7)


def test_norm_forward_is_torch_layer_norm():
    rng = np.random.default_rng(0)
    x, g, b = rng.standard_normal((5, 17)), rng.standard_normal(17), rng.standard_normal(17)
    ref = torch.nn.functional.layer_norm(torch.from_numpy(x), (17,), torch.from_numpy(g), torch.from_numpy(b), 1e-5)
    np.testing.assert_allclose(on.forward(x, g, b, 1e-5)[0], ref.numpy(), rtol=1e-12, atol=1e-13)


def test_topk_order_ties_masks_and_nan():
    nan, inf = np.nan, np.inf
    lg = np.array([[1.0, 3.0, 3.0, 2.0], [0.0, -0.0, -1.0, -inf], [-inf, -inf, 5.0, -inf], [-inf] * 4,
                   [1.0, nan, inf, nan]])
    assert ob.topk(lg, 3).tolist() == [[1, 2, 3], [0, 1, 2], [2, -1, -1], [-1, -1, -1], [1, 3, 2]]


def test_balance_loss_closed_forms():
    """Uniform logits and evenly used experts: balance = alpha exactly; one hot expert taking every slot's worth
    of probability: alpha E / K for K = 1."""
    T, E = 12, 6
    ids = (np.arange(T) % E).astype(np.int32)[:, None]
    r = ob.losses(np.zeros((T, E)), ids, 0.5, 0.25)
    np.testing.assert_allclose(r["loss"], [0.5, 0.25 * np.log(E) ** 2])
    hot = np.full((T, E), -50.0)
    hot[:, 2] = 50.0
    r = ob.losses(hot, np.full((T, 1), 2, dtype=np.int32), 0.5, 0.0)
    np.testing.assert_allclose(r["loss"][0], 0.5 * E)


@pytest.mark.parametrize("seg", [None, [0, 4, 4, 9], [1, 3, 8]])
def test_balance_gradient_by_differences(seg):
    rng = np.random.default_rng(3)
    T, E, K = 9, 5, 2
    lg = rng.standard_normal((T, E))
    lg[2, 1] = -np.inf
    lg[5] = -np.inf
    ids = ob.topk(lg, K, seg)
    counts = ob.losses(lg, ids, 0.3, 0.2, seg)["counts"]
    got = ob.gradient(lg, counts, K, 0.3, 0.2, (1.5, 0.5), seg)
    finite = np.isfinite(lg)

    def loss(v):
        full = np.where(finite, v, -np.inf)
        return np.dot([1.5, 0.5], ob.losses(full, ids, 0.3, 0.2, seg)["loss"])
    num = _fd(loss, np.where(finite, lg, 0.0))
    np.testing.assert_allclose(got, np.where(finite, num, 0.0), rtol=1e-6, atol=1e-8)


def test_sequences_are_independent_problems():
    """The packed loss is the token-weighted mean of the sequences' own losses."""
    rng = np.random.default_rng(4)
    lg = rng.standard_normal((10, 4))
    ids = ob.topk(lg, 2)
    whole = ob.losses(lg, ids, 1.0, 1.0, [0, 3, 10])["loss"]
    parts = [ob.losses(lg[a:b], ids[a:b], 1.0, 1.0)["loss"] * (b - a) / 10 for a, b in ((0, 3), (3, 10))]
    np.testing.assert_allclose(whole, sum(parts))


@pytest.mark.parametrize("values,byte,codes", [
    ([1.0, -0.5, 1 / 64, 1 / 128, 3 / 128], 121, [64, -32, 1, 0, 2]),   # ties to even: 0.5 -> 0, 1.5 -> 2
    ([1.9921875, -1.9921875], 121, [127, -127]),                        # 127.5 is clamped
    ([0.0, 0.0], 1, [0, 0]),
    ([2.0 ** -126], 1, [1]), ([2.0 ** -127], 1, [0]), ([1.5 * 2.0 ** -126], 1, [2]),
    ([2.0 ** 127], 248, [64]), ([np.inf], 255, None), ([np.nan, 1.0], 255, None),
])
def test_group_codes(values, byte, codes):
    v = np.zeros(32)
    v[:len(values)] = values
    c, b = oc.group_codes(v)
    assert b == byte
    if codes is not None:
        assert c[:len(codes)].tolist() == codes


def test_pack_error_bound_and_layout():
    rng = np.random.default_rng(5)
    ckpt = (rng.standard_normal((2, 2, 32, 256)) * np.exp(rng.standard_normal((2, 2, 32, 1)) * 4)).astype(np.float32)
    q, sf = oc.pack(ckpt)
    back = oc.unpack(q, sf)
    amax = np.abs(ckpt).reshape(2, 2, 32, 8, 32).max(-1, keepdims=True)
    err = np.abs(back - ckpt).reshape(2, 2, 32, 8, 32)
    assert np.all(err <= amax / 64)            # a step where the clamp acts, half of one elsewhere
    assert np.mean(err <= amax / 128) > 0.99
    assert torch.equal(torch.from_numpy(back).bfloat16().double(), torch.from_numpy(back))   # bf16 holds the values
    e = np.frexp(amax[..., 0])[1] - 1 + 127 - 6
    assert sf[1, 0, 1, 0, 2, 5] == e[1, 0, 5, 4 + 2]
