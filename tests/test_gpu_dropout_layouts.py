"""Dropout of the same rows wherever they lie: rows on and off the 16-byte boundary, of other strides than the result's, in few
and in many rows, give the same bits, by values in one rounding of the product and the sum."""
import numpy as np
import pytest
import torch

from helpers import np64
from oracle import dropout as od

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


def _at(t, shift, pad):
    """t's values in rows `pad` columns wider, the first `shift` elements behind a 16-byte boundary."""
    T, H = t.shape
    buf = torch.full((T * (H + pad) + shift,), float("nan"), dtype=t.dtype, device="cuda")
    out = buf[shift:].view(T, H + pad)[:, :H]
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(5, 64), (64, 1024), (40, 1111), (6000, 257)])
@pytest.mark.parametrize("residual", [True, False])
def test_same_bits_wherever_the_rows_lie(dtype, T, H, residual):
    mb = _mb()
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=gen, device="cuda").to(dtype)
    r = torch.randn(T, H, generator=gen, device="cuda").to(dtype) if residual else None
    ref = mb.dropout_fwd(x, 0.1, 5, 77, residual=r)
    for shift, pad in ((0, 8), (1, 0), (1, 7), (3, 5), (0, 1)):
        for which in ("both", "x", "r"):
            xs = x if which == "r" else _at(x, shift, pad)
            rs = r if which == "x" or not residual else _at(r, shift, pad)
            assert torch.equal(mb.dropout_fwd(xs, 0.1, 5, 77, residual=rs), ref), (shift, pad, which)
    assert torch.equal(mb.dropout_bwd(x, 0.1, 5, 77), mb.dropout_bwd(_at(x, 3, 5), 0.1, 5, 77))


@pytest.mark.parametrize("H", [512, 509])
def test_one_rounding(H):
    """fp32: the result is the exact sum with the factor as fp32 holds it, rounded once (half a step, 2^-24 of itself)."""
    mb = _mb()
    T, p = 50, 0.1
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(T, H, generator=gen, device="cuda") for _ in range(2))
    r = -x / (1 - p) * (1 + 1e-3 * r)          # sums that cancel: a product rounded by itself shows
    y = np64(mb.dropout_fwd(x, p, 5, 77, residual=r))
    keep = od.keep(T, H, p, 5, 77)
    ref = np64(r) + np.where(keep, np64(x) * float(np.float32(1 / (1 - p))), 0.0)
    assert np.all(np.abs(y - ref) <= U * np.abs(ref) * (1 + 2.0 ** -20))
