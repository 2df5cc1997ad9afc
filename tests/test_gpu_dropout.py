"""GPU parity of dropout_fwd / dropout_bwd: the mask bit for bit with the oracle's, values within their rounding, any width,
stride and alignment.

Bounds: x (1 / (1 - p)) in fp32 is two roundings of at most 2^-24 (the factor's and the product's), the sum with the residual
a third, relative to the magnitudes; the result is rounded to its type, by at most 2^-8 (bf16) of itself."""
import numpy as np
import pytest
import torch

from helpers import np64
from oracle import dropout as od

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SEED, OFFSET = 0x9D2C5680A7F13, (5 << 32) + 77


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


def _rand(T, H, dtype, seed, stride=None, shift=0):
    gen = torch.Generator().manual_seed(seed)
    stride = stride or H
    buf = torch.full((T * stride + shift,), float("nan"), dtype=dtype, device="cuda")
    out = buf[shift:shift + T * stride].view(T, stride)[:, :H] if T else buf[:0].view(0, H)
    v = torch.randn(T, H, generator=gen)
    v[v.abs() < 1e-3] = 1.0          # no zeros: what is dropped can be told from the result
    out.copy_(v.to(dtype))
    return out


def _bound(x, r, p, dtype, y):
    e = 4 * U * (np.abs(x) / (1 - p) + (0 if r is None else np.abs(r)))
    return e + (2.0 ** -8 if dtype == torch.bfloat16 else U) * (np.abs(y) + e)


CASES = [(1, 1), (1, 3), (2, 4), (3, 5), (7, 2048), (4, 1111), (33, 257), (5, 1024), (2, 6007), (700, 96), (64, 4097), (9000, 40)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", CASES)
@pytest.mark.parametrize("how", ["plain", "residual", "strided", "shifted"])
def test_forward(dtype, T, H, how):
    mb = _mb()
    p = 0.1 + 0.05 * (H % 7)
    x = _rand(T, H, dtype, 1, H + 24 if how == "strided" else H + 5 if how == "shifted" else None, 3 if how == "shifted" else 0)
    r = None if how == "plain" else _rand(T, H, dtype, 2, H + 8 if how == "strided" else None)
    y = mb.dropout_fwd(x, p, SEED, OFFSET, residual=r)
    torch.cuda.synchronize()
    xs, rs = np64(x), None if r is None else np64(r)
    ref = od.forward(xs, p, SEED, OFFSET, rs)
    assert y.shape == (T, H) and y.dtype == dtype
    assert np.all(np.abs(np64(y) - ref) <= _bound(xs, rs, p, dtype, ref))
    if r is None:
        assert np.array_equal(np64(y) != 0, od.keep(T, H, p, SEED, OFFSET))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(3, 5), (33, 257), (40, 512), (4000, 333)])
def test_backward_has_the_forwards_mask(dtype, T, H):
    """dx of <dy, y> by differences: y is linear in x, so y(x + d) - y(x) = keep d / (1 - p) and dx = keep dy / (1 - p)."""
    mb = _mb()
    dy = _rand(T, H, dtype, 3, H + 2)
    dx = mb.dropout_bwd(dy, 0.3, SEED, OFFSET)
    y = mb.dropout_fwd(torch.ones_like(dx), 0.3, SEED, OFFSET)
    torch.cuda.synchronize()
    assert torch.equal(dx != 0, y != 0)
    ref = od.forward(np64(dy), 0.3, SEED, OFFSET)
    assert np.all(np.abs(np64(dx) - ref) <= _bound(np64(dy), None, 0.3, dtype, ref))


def test_mask_is_a_function_of_position_alone():
    mb = _mb()
    x = torch.ones(50, 1111, device="cuda")
    full = mb.dropout_fwd(x, 0.4, 1, 2)
    assert torch.equal(mb.dropout_fwd(x[:20], 0.4, 1, 2), full[:20])
    assert torch.equal(mb.dropout_fwd(x[:, :300], 0.4, 1, 2), full[:, :300])
    assert torch.equal(mb.dropout_fwd(x.bfloat16(), 0.4, 1, 2) != 0, full != 0)
    dev = torch.tensor([2], dtype=torch.int64, device="cuda")
    assert torch.equal(mb.dropout_fwd(x, 0.4, 1, dev), full)
    for other in (mb.dropout_fwd(x, 0.4, 2, 2), mb.dropout_fwd(x, 0.4, 1, 3), mb.dropout_fwd(x, 0.4, 1 + 2 ** 40, 2)):
        assert not torch.equal(other, full)


def test_no_dropping_and_nearly_all():
    mb = _mb()
    x, r = _rand(5, 77, torch.float32, 1), _rand(5, 77, torch.float32, 2)
    assert torch.equal(mb.dropout_fwd(x, 0.0, 3), x) and torch.equal(mb.dropout_fwd(x, 0.0, 3, residual=r), x + r)
    assert torch.equal(mb.dropout_fwd(x, 1 - 2.0 ** -40, 3, residual=r), r)
    e = mb.dropout_fwd(x[:0], 0.5, 3)
    assert e.shape == (0, 77)


def test_dropped_values_are_gone():
    """Infinities and NaN in dropped places leave no trace; in kept places they stay."""
    mb = _mb()
    m = torch.from_numpy(od.keep(6, 203, 0.5, 4, 0)).cuda()
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.where(m, 2.0, bad).float()
        y = mb.dropout_fwd(x, 0.5, 4, residual=torch.ones_like(x))
        assert torch.equal(y, torch.where(m, 5.0, 1.0))
        assert torch.all(~torch.isfinite(mb.dropout_fwd(torch.full_like(x, bad), 0.5, 4)[m]))


def test_in_place_and_bounds_of_rows():
    """y may be x or the residual; nothing outside the rows is written."""
    mb = _mb()
    lib = mb.lib()
    T, H = 9, 205
    for dtype, code in ((torch.bfloat16, 0), (torch.float32, 1)):
        for which in ("x", "residual"):
            buf = torch.full((T * H + 64,), 7.0, dtype=dtype, device="cuda")
            other = _rand(T, H, dtype, 5)
            inside = buf[32:32 + T * H].view(T, H)
            inside.copy_(_rand(T, H, dtype, 6))
            x, r = (inside, other) if which == "x" else (other, inside)
            ref = mb.dropout_fwd(x, 0.25, 9, 1, residual=r)
            st = torch.cuda.current_stream().cuda_stream
            assert lib.dropout_fwd(x.data_ptr(), H, r.data_ptr(), H, code, T, H, 0.25, 9, 1, None, inside.data_ptr(), st) == 0
            torch.cuda.synchronize()
            assert torch.equal(inside, ref) and torch.all(buf[:32] == 7) and torch.all(buf[32 + T * H:] == 7)


def test_graph_takes_new_offsets():
    """A captured call with the offset on the device draws a new mask at every replay."""
    mb = _mb()
    x = torch.ones(64, 130, device="cuda")
    at = torch.zeros(1, dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    mb.dropout_fwd(x, 0.5, 11, at)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y = mb.dropout_fwd(x, 0.5, 11, at)
        dx = mb.dropout_bwd(x, 0.5, 11, at)
        at += 1
    for step in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, mb.dropout_fwd(x, 0.5, 11, step)) and torch.equal(y, dx)


def test_streams():
    mb = _mb()
    x = _rand(100, 333, torch.bfloat16, 1)
    ref = mb.dropout_fwd(x, 0.2, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = mb.dropout_fwd(x, 0.2, 5, stream=side)
    side.synchronize()
    assert torch.equal(ref, y)


def test_past_32_bits():
    """The last rows of a tensor of more than 2^31 elements."""
    mb = _mb()
    H = 4099
    T = 2 ** 31 // H + 40
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    y = mb.dropout_fwd(x, 0.5, 8, residual=x)
    torch.cuda.synchronize()
    m = torch.from_numpy(od.keep(8, H, 0.5, 8, 0, row0=T - 8)).cuda()
    assert torch.equal(y[T - 8:], torch.where(m, 3.0, 1.0).bfloat16())


def test_refusals():
    mb = _mb()
    x = torch.ones(4, 64, device="cuda")
    for args, kw in (((x.cpu(), 0.5, 1), {}), ((x.half(), 0.5, 1), {}), ((x[0], 0.5, 1), {}), ((x[:, ::2], 0.5, 1), {}),
                     ((x, 1.0, 1), {}), ((x, -0.1, 1), {}), ((x, float("nan"), 1), {}), ((x, 0.5, -1), {}), ((x, 0.5, 2 ** 64), {}),
                     ((x, 0.5, 1, -1), {}), ((x, 0.5, 1, torch.zeros(1, device="cuda")), {}),
                     ((x, 0.5, 1), dict(residual=x.bfloat16())), ((x, 0.5, 1), dict(residual=x[:2]))):
        with pytest.raises(mb.MoeError):
            mb.dropout_fwd(*args, **kw)
