"""GPU parity of layer_norm_fwd / layer_norm_bwd against the float64 oracle: both kinds, types and weight types,
widths that are odd, below a warp and above a block, row strides, unaligned rows, a single row, none, one column,
the residual and the skip gradient.

Bounds: u = 2^-24 is fp32's rounding unit and a sum of H terms in any order is off by at most H u times the sum
of magnitudes, so with the row's mean and rstd each carrying H u (1 + mean|s| rstd), every intermediate is off
by at most (4 H + 64) u (1 + mean|s| rstd) times the sum of the magnitudes it is made of; the result is then
rounded to its type, by at most 2^-8 (bf16) or u (fp32) of itself."""
import numpy as np
import pytest
import torch

from helpers import np64
from oracle import norm as on

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


def _rand(shape, dtype, seed, stride=None, shift=0):
    """Rows on the GPU; stride: elements from row to row; shift: elements off the allocation's start."""
    gen = torch.Generator().manual_seed(seed)
    T, H = shape
    v = torch.randn(T, H, generator=gen).to(dtype)
    stride = stride or H
    buf = torch.full((T * stride + shift,), float("nan"), dtype=dtype, device="cuda")
    out = buf[shift:shift + T * stride].view(T, stride)[:, :H] if T else buf[:0].view(0, H)
    out.copy_(v)
    return out


def _unit(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


CASES = [(1, 1), (1, 2048), (3, 7), (5, 64), (2, 100), (4, 1111), (3, 1024), (2, 4096), (2, 5000), (3, 8192), (2, 12288),
         (70, 256), (333, 96), (150, 520)]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", CASES)
@pytest.mark.parametrize("how", ["plain", "residual", "strided"])
def test_forward(kind, dtype, T, H, how):
    mb = _mb()
    wt = torch.float32 if (T + H) % 2 else torch.bfloat16
    strided = how == "strided"
    x = _rand((T, H), dtype, 1, H + 24 if strided else None, 1 if strided else 0)
    x += 0.5
    r = _rand((T, H), dtype, 2, H + 3 if strided else None) if how != "plain" else None
    gamma, beta = _rand((1, H), wt, 3)[0], _rand((1, H), wt, 4)[0]
    out = mb.layer_norm_fwd(x, gamma, beta if how != "strided" else None, eps=EPS, residual=r, kind=kind)
    torch.cuda.synchronize()
    s = x if r is None else (x.float() + r.float()).to(dtype)
    if r is not None:
        assert torch.equal(out["sum"], s)
    else:
        assert out["sum"] is None
    b = None if strided else np64(beta)
    y, mean, rstd = on.forward(np64(s), np64(gamma), b, EPS, kind)
    grow = (4 * H + 64) * U * (1 + np.abs(np64(s)).mean(1) * rstd)
    assert np.all(np.abs(np64(out["rstd"]) - rstd) <= grow * rstd)
    if kind == 0:
        assert np.all(np.abs(np64(out["mean"]) - mean) <= H * U * np.abs(np64(s)).mean(1) + U * np.abs(mean))
    else:
        assert out["mean"] is None
    parts = (np.abs(np64(s)) + np.abs(mean)[:, None]) * rstd[:, None] * np.abs(np64(gamma))
    bound = grow[:, None] * (parts + (0 if b is None else np.abs(b))) + _unit(dtype) * np.abs(y)
    assert np.all(np.abs(np64(out["y"]) - y) <= bound)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", CASES)
@pytest.mark.parametrize("how", ["plain", "skip", "strided"])
def test_backward(kind, dtype, T, H, how):
    if H > 6000:
        T = 1          # the oracle's Jacobian is H x H
    mb = _mb()
    wt = torch.float32 if (T + H) % 2 else torch.bfloat16
    strided = how == "strided"
    x = _rand((T, H), dtype, 1, H + 24 if strided else None, 1 if strided else 0)
    x += 0.25
    dy = _rand((T, H), dtype, 5, H + 8 if strided else None)
    dres = _rand((T, H), dtype, 6, H + 5 if strided else None) if how != "plain" else None
    gamma = _rand((1, H), wt, 3)[0]
    xs, dys, g = np64(x), np64(dy), np64(gamma)
    _, mean, rstd = on.forward(xs, g, None, EPS, kind)
    f32 = lambda v: torch.from_numpy(v).float().cuda()  # noqa: E731
    out = mb.layer_norm_bwd(dy, x, gamma, f32(mean) if kind == 0 else None, f32(rstd), dres=dres, kind=kind)
    torch.cuda.synchronize()
    dx, dg, db = on.backward(dys, xs, g, EPS, kind, None if dres is None else np64(dres))
    w, xh = dys * g, (xs - mean[:, None]) * rstd[:, None]
    grow = ((4 * H + 64) * U * (1 + np.abs(xs).mean(1) * rstd))[:, None]
    parts = rstd[:, None] * (np.abs(w) + np.abs(w).mean(1, keepdims=True)
                             + (np.abs(xh) + 1) * np.abs(w * xh).mean(1, keepdims=True))
    if dres is not None:
        parts = parts + np.abs(np64(dres))
    assert np.all(np.abs(np64(out["dx"]) - dx) <= grow * parts + _unit(dtype) * np.abs(dx))
    rows = (T + 64) * U + 8 * U * (1 + np.abs(mean) * rstd).max()
    assert np.all(np.abs(np64(out["dgamma"]) - dg) <= rows * (np.abs(dys) * (np.abs(xh) + 1)).sum(0))
    if kind == 0:
        assert np.all(np.abs(np64(out["dbeta"]) - db) <= (T + 64) * U * np.abs(dys).sum(0))
    else:
        assert out["dbeta"] is None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,pad,shift", [(5000, 200, 0, 0), (9001, 333, 0, 0), (4100, 1001, 3, 0), (3000, 1536, 8, 0),
                                           (2500, 2049, 0, 0), (1300, 4095, 0, 0), (900, 6001, 1, 0), (3000, 771, 5, 1), (4001, 601, 0, 0)])
def test_many_rows(dtype, T, H, pad, shift):
    """Many rows per block: every slot of the ring is filled again several times, in each way of reading rows
    (vectors, rows that begin anywhere in a 16-byte piece, an unaligned base).  Against torch's float64 layer norm
    and its automatic differentiation, with the bounds above."""
    mb = _mb()
    x, r, dy, dres = (_rand((T, H), dtype, k, H + pad, shift) for k in (1, 2, 5, 6))
    gamma, beta = _rand((1, H), torch.float32, 3)[0], _rand((1, H), torch.float32, 4)[0]
    f = mb.layer_norm_fwd(x, gamma, beta, eps=EPS, residual=r)
    b = mb.layer_norm_bwd(dy, f["sum"], gamma, f["mean"], f["rstd"], dres=dres)
    assert torch.equal(f["sum"], (x.float() + r.float()).to(dtype))
    s64, g64, b64 = f["sum"].double().requires_grad_(), gamma.double().requires_grad_(), beta.double().requires_grad_()
    y = torch.nn.functional.layer_norm(s64, (H,), g64, b64, EPS)
    (y * dy.double()).sum().backward()
    grow = (4 * H + 64) * U * 2
    y, d = y.detach(), s64.grad + dres.double()
    xh = (s64.detach() - f["mean"].double()[:, None]) * f["rstd"].double()[:, None]
    assert torch.all((f["y"].double() - y).abs() <= grow * (xh.abs() * gamma.abs() + beta.abs() + 1) + _unit(dtype) * y.abs())
    w = (dy.double() * gamma).abs()
    parts = f["rstd"].double()[:, None] * (w + w.mean(1, keepdim=True) + (xh.abs() + 1) * (w * xh.abs()).mean(1, keepdim=True))
    assert torch.all((b["dx"].double() - d).abs() <= grow * (parts + dres.double().abs()) + _unit(dtype) * d.abs())
    rows = (T + 64) * U
    assert torch.all((b["dgamma"].double() - g64.grad).abs() <= 2 * rows * (dy.double().abs() * (xh.abs() + 1)).sum(0))
    assert torch.all((b["dbeta"].double() - b64.grad).abs() <= rows * dy.double().abs().sum(0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_mean_and_constant_rows(dtype):
    """The variance is of differences from the mean: rows far from zero keep it, a constant row has rstd
    1 / sqrt(eps) and y = beta."""
    mb = _mb()
    H = 512
    x = torch.full((2, H), 96.0, dtype=dtype, device="cuda")
    x[1, ::2] += 1.0    # exact in bf16: 96 and 97, variance 1/4
    one, zero = torch.ones(H, device="cuda"), torch.zeros(H, device="cuda")
    out = mb.layer_norm_fwd(x, one, zero + 3, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(out["y"][0].float(), torch.full((H,), 3.0, device="cuda"))
    np.testing.assert_allclose(np64(out["rstd"]), [EPS ** -0.5, (0.25 + EPS) ** -0.5], rtol=1e-5)
    assert np64(out["mean"]).tolist() == [96.0, 96.5]


def test_gradient_against_differences_of_the_forward():
    """dx by central differences of the GPU's own fp32 forward: step 2^-6, so rounding is about 2^-24 sqrt(H) |y|
    / 2^-6 ~ 1e-4 of the gradient's scale and truncation about 2^-12."""
    mb = _mb()
    T, H = 3, 24
    x, dy, gamma, beta = (_rand((t, H), torch.float32, k) for t, k in ((T, 1), (T, 2), (1, 3), (1, 4)))
    gamma, beta = gamma[0], beta[0]
    f = mb.layer_norm_fwd(x, gamma, beta, eps=1e-2)
    g = np64(mb.layer_norm_bwd(dy, x, gamma, f["mean"], f["rstd"])["dx"])
    h = 2.0 ** -6
    num = np.zeros((T, H))
    for i in range(H):
        d = torch.zeros(T, H, device="cuda")
        d[:, i] = h
        y1, y0 = (mb.layer_norm_fwd(x + s * d, gamma, beta, eps=1e-2)["y"] for s in (1, -1))
        num[:, i] = ((np64(y1) - np64(y0)) * np64(dy)).sum(1) / (2 * h)
    assert np.abs(num - g).max() <= 2e-3 * np.abs(g).max()


def test_accumulate_repeats_and_streams():
    """dgamma and dbeta added to an earlier result; the same call twice, and on another stream, gives the same bits."""
    mb = _mb()
    T, H = 1000, 384
    x, dy = _rand((T, H), torch.bfloat16, 1), _rand((T, H), torch.bfloat16, 2)
    gamma = torch.ones(H, device="cuda")
    f = mb.layer_norm_fwd(x, gamma, gamma)
    a = mb.layer_norm_bwd(dy, x, gamma, f["mean"], f["rstd"])
    ga, ba = a["dgamma"].clone(), a["dbeta"].clone()
    mb.layer_norm_bwd(dy, x, gamma, f["mean"], f["rstd"], accumulate_into=a)
    torch.cuda.synchronize()
    assert torch.equal(a["dgamma"], ga + ga) and torch.equal(a["dbeta"], ba + ba)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = mb.layer_norm_bwd(dy, x, gamma, f["mean"], f["rstd"], stream=side)
    side.synchronize()
    for k in ("dx",):
        assert torch.equal(b[k], a[k])
    assert torch.equal(b["dgamma"], ga) and torch.equal(b["dbeta"], ba)


@pytest.mark.parametrize("T,H", [(5, 640), (700, 333), (2000, 2048)])
def test_residual_stream_updated_in_place(T, H):
    """sum may be x or the residual themselves (C entry point)."""
    mb = _mb()
    x, r = _rand((T, H), torch.bfloat16, 1), _rand((T, H), torch.bfloat16, 2)
    gamma = torch.ones(H, device="cuda")
    ref = mb.layer_norm_fwd(x, gamma, gamma, residual=r)
    for target in (x.clone(), r.clone()):
        xx, rr = (target, r) if torch.equal(target, x) else (x, target)
        y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        rc = mb.lib().layer_norm_fwd(0, xx.data_ptr(), H, rr.data_ptr(), H, gamma.data_ptr(), gamma.data_ptr(), 0, 1, T, H,
                                     1e-5, y.data_ptr(), target.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal(target, ref["sum"]) and torch.equal(y, ref["y"])


def test_empty_and_refusals():
    mb = _mb()
    g = torch.ones(8, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    z = torch.empty(0, device="cuda")
    assert mb.layer_norm_fwd(e, g)["y"].shape == (0, 8)
    out = mb.layer_norm_bwd(e, e, g, z, z)
    torch.cuda.synchronize()
    assert not out["dgamma"].any() and not out["dbeta"].any()
    x = torch.ones(2, 8, device="cuda")
    s = torch.ones(2, device="cuda")
    for bad in (lambda: mb.layer_norm_fwd(x.half(), g), lambda: mb.layer_norm_fwd(x, g[:7]),
                lambda: mb.layer_norm_fwd(x.t(), torch.ones(2, device="cuda")), lambda: mb.layer_norm_fwd(x.cpu(), g),
                lambda: mb.layer_norm_fwd(x, g, residual=x[:1]), lambda: mb.layer_norm_fwd(x, g, eps=-1.0),
                lambda: mb.layer_norm_fwd(x[:1].expand(2, 8), g), lambda: mb.layer_norm_fwd(x, g, kind=2),
                lambda: mb.layer_norm_bwd(x.bfloat16(), x, g, s, s), lambda: mb.layer_norm_bwd(x, x, g, s[:1], s),
                lambda: mb.layer_norm_bwd(x, x, g, None, s)):
        with pytest.raises(mb.MoeError):
            bad()


@pytest.mark.parametrize("T", [1, 7, 300])
@pytest.mark.parametrize("H,shift", [(96, 0), (1111, 0), (2048, 0), (2048, 1)])
def test_calls_back_to_back_on_reused_buffers(T, H, shift):
    """A kernel may start before the one in front of it has written: forward and backward one right after the other on the
    same statistics buffers, and a norm's output as the next norm's weights, with other inputs each time, give the
    bits of calls that are waited for one by one."""
    mb = _mb()
    n = 40
    lib, st = mb.lib(), torch.cuda.current_stream().cuda_stream
    x, dy = ([_rand((T, H), torch.float32, 100 * k + i, None, shift) for i in range(n)] for k in (1, 2))
    z = [_rand((1, H), torch.float32, 300 + i) for i in range(n)]
    gamma = _rand((1, H), torch.float32, 4)[0]
    size = max(lib.layer_norm_bwd_workspace_size(T, H), 256)

    def run(wait):
        new = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        y, w, mean, rstd, m1, r1, ws = new(T, H), new(1, H), new(T), new(T), new(1), new(1), new(size // 4)
        m2, r2 = new(T), new(T)
        dx, dg, db, y2 = new(n, T, H), new(n, H), new(n, H), new(n, T, H)
        torch.cuda.synchronize()
        for i in range(n):
            calls = [lambda: lib.layer_norm_fwd(0, x[i].data_ptr(), H, None, 0, gamma.data_ptr(), None, 1, 1, T, H, EPS,
                                                y.data_ptr(), None, mean.data_ptr(), rstd.data_ptr(), st),
                     lambda: lib.layer_norm_bwd(0, dy[i].data_ptr(), H, x[i].data_ptr(), H, gamma.data_ptr(), mean.data_ptr(),
                                                rstd.data_ptr(), None, 0, 1, 1, T, H, dx[i].data_ptr(), dg[i].data_ptr(),
                                                db[i].data_ptr(), 0, ws.data_ptr(), size, st),
                     lambda: lib.layer_norm_fwd(0, z[i].data_ptr(), H, None, 0, gamma.data_ptr(), None, 1, 1, 1, H, EPS,
                                                w.data_ptr(), None, m1.data_ptr(), r1.data_ptr(), st),
                     lambda: lib.layer_norm_fwd(0, x[i].data_ptr(), H, None, 0, w.data_ptr(), w.data_ptr(), 1, 1, T, H, EPS,
                                                y2[i].data_ptr(), None, m2.data_ptr(), r2.data_ptr(), st)]
            for call in calls:
                assert call() == 0
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return dx, dg, db, y2

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,pad,shift", [(700, 8200, 0, 0), (333, 12288, 8, 0), (97, 16385, 0, 1), (40, 32768, 0, 0)])
def test_many_wide_rows(dtype, T, H, pad, shift):
    """Above 8192 columns: several row groups, several rows a warp of a group, column tiles that end inside 32."""
    test_many_rows(dtype, T, H, pad, shift)


@pytest.mark.parametrize("H", [8200, 1024])
def test_root_mean_square_over_many_rows(H):
    """The form without a mean: dx and dgamma against automatic differentiation of its formula in float64; dgamma added to
    an earlier result."""
    mb = _mb()
    T = 650
    x, dy, dres = (_rand((T, H), torch.float32, k) for k in (1, 5, 6))
    gamma = _rand((1, H), torch.float32, 3)[0]
    f = mb.layer_norm_fwd(x, gamma, None, eps=EPS, kind=1)
    b = mb.layer_norm_bwd(dy, x, gamma, None, f["rstd"], dres=dres, kind=1)
    x64, g64 = x.double().requires_grad_(), gamma.double().requires_grad_()
    y = x64 * (x64.square().mean(-1, keepdim=True) + EPS).rsqrt() * g64
    (y * dy.double()).sum().backward()
    grow = (4 * H + 64) * U * 2
    y, d = y.detach(), x64.grad + dres.double()
    xh = x.double() * f["rstd"].double()[:, None]
    assert torch.all((f["y"].double() - y).abs() <= grow * xh.abs() * gamma.abs().double() + U * y.abs())
    w = (dy.double() * gamma).abs()
    parts = f["rstd"].double()[:, None] * (w + xh.abs() * (w * xh.abs()).mean(1, keepdim=True))
    assert torch.all((b["dx"].double() - d).abs() <= grow * (parts + dres.double().abs()) + U * d.abs())
    size = (dy.double().abs() * xh.abs()).sum(0)
    assert torch.all((b["dgamma"].double() - g64.grad).abs() <= (2 * (T + 64) * U + grow) * size)
    before = b["dgamma"].clone()
    mb.layer_norm_bwd(dy, x, gamma, None, f["rstd"], dres=dres, kind=1, accumulate_into=b)
    assert b["dbeta"] is None and torch.equal(b["dgamma"], before + before)
