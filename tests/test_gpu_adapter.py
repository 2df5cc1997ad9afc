"""GPU parity of adapter_fwd / adapter_bwd against the float64 oracle: ranks and widths off the tiles, one token to thousands,
adapters without a token, tokens without an adapter, strided rows, in place, accumulation, graphs, wrong metadata.

Bounds, elementwise.  u = 2^-24; a product of K terms summed in fp32 in any order (truncating adds counted: 2 u) is off by at
most e(K) = 2 (K + 8) u times the sum of the terms' magnitudes.  Every rounding to bf16 is off by at most 2^-8 of the value."""
import numpy as np
import pytest
import torch

from helpers import np64
from oracle import adapter as oa

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


def _e(K):
    return 2 * (K + 8) * U


def _inputs(T, H, N, n, r, seed=0, none=0.2, only=None, strided=False):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    bf = torch.bfloat16
    ids = torch.randint(0, n, (T,), generator=gen)
    if only is not None:
        ids = torch.tensor(only)[torch.randint(0, len(only), (T,), generator=gen)]
    ids[torch.rand(T, generator=gen) < none] = -1
    d = dict(x=rand(T, H).to(bf), dy=rand(T, N).to(bf), A=(rand(n, r, H) * H ** -0.5).to(bf), B=(rand(n, r, N) * r ** -0.5).to(bf),
             scale=0.5 + torch.rand(n, generator=gen), base=rand(T, N).to(bf), dbase=rand(T, H).to(bf),
             ids=ids.to(torch.int32)[:, None].contiguous())
    d = {k: v.cuda() for k, v in d.items()}
    if strided:
        for k, pad in (("x", 24), ("dy", 8), ("base", 16), ("dbase", 8)):
            wide = torch.full((T, d[k].shape[1] + pad), float("nan"), dtype=bf, device="cuda")
            wide[:, : d[k].shape[1]] = d[k]
            d[k] = wide[:, : d[k].shape[1]]
    d["meta"] = _mb().route_meta(d["ids"], n, 128)
    return d


def _sel(d):
    ids = d["ids"].cpu().numpy()[:, 0]
    have = (ids >= 0)[:, None]
    i = np.maximum(ids, 0)
    return ids, have, i


def _check_fwd(d, got, base="base"):
    ids, have, i = _sel(d)
    x, A, B, scale = (np64(d[k]) for k in ("x", "A", "B", "scale"))
    b = np64(d[base]) if base else np.zeros((x.shape[0], B.shape[2]))
    y, u = oa.forward(x, A, B, ids, scale, b)
    H, r = x.shape[1], A.shape[1]
    eu = np.zeros_like(u)
    ey = np.zeros_like(y)
    for t in np.flatnonzero(have[:, 0]):
        a = ids[t]
        eu[t] = _e(H) * (np.abs(A[a]) @ np.abs(x[t]))
        su = scale[a] * (np.abs(u[t]) + eu[t])
        ev = scale[a] * eu[t] + (HALF + 2 * U) * su
        ey[t] = ev @ np.abs(B[a]) + _e(r + 1) * ((su + ev) @ np.abs(B[a]) + np.abs(b[t]))
    if got["u"] is not None:
        assert np.all(np.abs(np64(got["u"]) - u) <= eu)
    assert np.all(np.abs(np64(got["y"]) - y) <= ey + HALF * (np.abs(y) + ey) * have)


def _check_bwd(d, u, got, base="dbase", times=1):
    ids, have, i = _sel(d)
    x, dy, A, B, scale, uu = (np64(v) for v in (d["x"], d["dy"], d["A"], d["B"], d["scale"], u))
    b = np64(d[base]) if base else np.zeros_like(x)
    dx, dA, dB = oa.backward(dy, x, uu, A, B, ids, scale, b)
    N, r = dy.shape[1], A.shape[1]
    edx, edA, edB = np.zeros_like(dx), np.zeros_like(dA), np.zeros_like(dB)
    for a in range(A.shape[0]):
        rows = np.flatnonzero(ids == a)
        m = scale[a] * (np.abs(dy[rows]) @ np.abs(B[a]).T)
        v = np.abs(scale[a] * (dy[rows] @ B[a].T))
        ev = _e(N + 1) * m
        ev = ev + HALF * (v + ev)
        edx[rows] = ev @ np.abs(A[a]) + _e(r + 1) * ((v + ev) @ np.abs(A[a]) + np.abs(b[rows]))
        k = _e(len(rows) + 8)
        edA[a] = ev.T @ np.abs(x[rows]) + k * ((v + ev).T @ np.abs(x[rows]))
        s = scale[a] * np.abs(uu[rows])
        es = (HALF + 2 * U) * s
        edB[a] = es.T @ np.abs(dy[rows]) + k * ((s + es).T @ np.abs(dy[rows]))
    assert np.all(np.abs(np64(got["dx"]) - dx) <= edx + HALF * (np.abs(dx) + edx) * have)
    for n, ref, e in (("dA", dA, edA), ("dB", dB, edB)):
        e = e + HALF * (np.abs(ref) + e)
        if times == 2:          # added onto an earlier, rounded result
            ref, e = 2 * ref, 2 * e + HALF * (2 * np.abs(ref) + 2 * e)
        assert np.all(np.abs(np64(got[n]) - ref) <= e), n


# T, H, N, n, r
CASES = [(1, 8, 8, 1, 1), (1, 512, 264, 3, 16), (7, 64, 72, 4, 4), (48, 1024, 512, 32, 16), (63, 136, 8, 2, 5), (64, 128, 128, 1, 8),
         (65, 200, 1000, 1, 17), (130, 520, 392, 5, 32), (300, 1000, 1240, 7, 12), (513, 264, 136, 3, 64), (700, 72, 648, 40, 128),
         (1300, 136, 264, 2, 33)]


@pytest.mark.parametrize("T,H,N,n,r", CASES)
@pytest.mark.parametrize("how", ["plain", "strided", "bare"])
def test_forward_and_backward(T, H, N, n, r, how):
    mb = _mb()
    d = _inputs(T, H, N, n, r, seed=T + r, none=0.0 if T == 1 else 0.2, strided=how == "strided")
    if how == "bare":
        d["scale"] = torch.ones(n, device="cuda")
        f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"])
        g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"])
        torch.cuda.synchronize()
        _check_fwd(d, f, None)
        _check_bwd(d, f["u"], g, None)
        return
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])
    torch.cuda.synchronize()
    _check_fwd(d, f)
    _check_bwd(d, f["u"], g)


@pytest.mark.parametrize("T", [700, 5000, 9000])
def test_long_groups(T):
    """Adapters with more rows than one gradient tile next to ones with few and none."""
    mb = _mb()
    d = _inputs(T, 136, 72, 6, 20, seed=T, none=0.1, only=[0, 0, 0, 0, 0, 0, 0, 0, 3, 3, 3, 3, 3, 3, 5])
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])
    torch.cuda.synchronize()
    _check_fwd(d, f)
    _check_bwd(d, f["u"], g)
    assert torch.all(g["dA"][[1, 2, 4]] == 0) and torch.all(g["dB"][[1, 2, 4]] == 0)
    again = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])
    torch.cuda.synchronize()
    assert all(torch.equal(g[k], again[k]) for k in g)
    more = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"], accumulate_into=again)
    torch.cuda.synchronize()
    assert more["dA"] is again["dA"]
    _check_bwd(d, f["u"], more, times=2)


def test_no_adapter_at_all_and_no_rows():
    mb = _mb()
    d = _inputs(70, 64, 136, 3, 8, none=1.1)
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])
    torch.cuda.synchronize()
    assert torch.equal(f["y"], d["base"]) and torch.all(f["u"] == 0) and torch.equal(g["dx"], d["dbase"])
    assert torch.all(g["dA"] == 0) and torch.all(g["dB"] == 0)
    e = {k: v[:0] for k, v in d.items() if k in ("x", "dy", "base", "dbase")}
    meta = dict(expert_offsets=torch.zeros(4, dtype=torch.int32, device="cuda"),
                x_gather_idx=torch.zeros(0, dtype=torch.int32, device="cuda"),
                s_reverse_scatter_idx=torch.zeros(0, dtype=torch.int32, device="cuda"))
    f = mb.adapter_fwd(e["x"], d["A"], d["B"], meta, base=e["base"])
    g = mb.adapter_bwd(e["dy"], e["x"], f["u"], d["A"], d["B"], meta, base=e["dbase"])
    torch.cuda.synchronize()
    assert f["y"].shape == (0, 136) and torch.all(g["dA"] == 0) and torch.all(g["dB"] == 0)


def test_in_place():
    """The adapters' part added onto the shared projection's own output."""
    mb = _mb()
    d = _inputs(200, 136, 520, 4, 16)
    ref = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    g = mb.adapter_bwd(d["dy"], d["x"], ref["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])
    y, dx = d["base"].clone(), d["dbase"].clone()
    f2 = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=y, out=y, save=False)
    g2 = mb.adapter_bwd(d["dy"], d["x"], ref["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=dx, out=dx)
    torch.cuda.synchronize()
    assert f2["y"] is y and f2["u"] is None and torch.equal(y, ref["y"])
    assert g2["dx"] is dx and torch.equal(dx, g["dx"])


def test_rows_do_not_depend_on_the_batch():
    mb = _mb()
    d = _inputs(40, 256, 136, 4, 16, none=0.0)
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    part = mb.route_meta(d["ids"][10:21].contiguous(), 4, 128)
    p = mb.adapter_fwd(d["x"][10:21], d["A"], d["B"], part, scale=d["scale"], base=d["base"][10:21])
    torch.cuda.synchronize()
    assert torch.equal(f["y"][10:21], p["y"])


def test_beside_a_shared_projection():
    """A fine-tuning step of one linear layer: Y = X W^T with adapters on top, linear_bwd, the adapters' gradients onto its dX."""
    mb = _mb()
    T, H, N, n, r = 384, 256, 128, 3, 16
    d = _inputs(T, H, N, n, r, seed=5)
    W = (torch.randn(N, H, generator=torch.Generator().manual_seed(1)) * H ** -0.5).to(torch.bfloat16).cuda()
    y = d["x"] @ W.t()
    d["base"] = y.clone()
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=y, out=y)
    lin = mb.linear_bwd(d["dy"], W, d["x"], precision=mb.PREC_BF16)
    d["dbase"] = lin["dX"].clone()
    g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=lin["dX"], out=lin["dX"])
    torch.cuda.synchronize()
    _check_fwd(d, f)
    _check_bwd(d, f["u"], g)


def test_streams_and_graph():
    mb = _mb()
    d = _inputs(150, 136, 264, 5, 24)

    def calls(stream=None):
        meta = mb.route_meta(d["ids"], 5, 128, stream=stream)
        f = mb.adapter_fwd(d["x"], d["A"], d["B"], meta, scale=d["scale"], base=d["base"], stream=stream)
        g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], meta, scale=d["scale"], base=d["dbase"], stream=stream)
        return [f["y"], f["u"], g["dx"], g["dA"], g["dB"]]

    ref = calls()
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        h1 = calls()
    with torch.cuda.graph(g2):
        h2 = calls()
    d["x"].mul_(-0.5)
    d["ids"].copy_(d["ids"].flip(0))          # the metadata is captured with the calls
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    now = calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(now, h1, h2))
    assert not torch.equal(now[0], ref[0])


def test_infinities_stay_in_their_rows():
    mb = _mb()
    d = _inputs(100, 64, 72, 2, 8, none=0.3)
    d["x"][17] = float("inf")
    d["x"][18] = float("nan")
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    torch.cuda.synchronize()
    bad = ~torch.isfinite(f["y"]).all(1)
    have = d["ids"][:, 0] >= 0
    want = torch.zeros_like(bad)
    want[17], want[18] = have[17], have[18]
    assert torch.equal(bad, want)


def test_refusals():
    mb = _mb()
    d = _inputs(16, 64, 72, 2, 8)
    f = lambda **k: mb.adapter_fwd(**{**dict(x=d["x"], A=d["A"], B=d["B"], route_meta=d["meta"], scale=d["scale"], base=d["base"]), **k})  # noqa: E731
    other = mb.route_meta(d["ids"], 3, 128)
    for bad in (dict(x=d["x"].cpu()), dict(x=d["x"].float()), dict(A=d["A"][:1]), dict(A=d["A"].transpose(1, 2)), dict(B=d["B"].float()),
                dict(scale=d["scale"].double()), dict(base=d["base"][:, :64]), dict(route_meta=other), dict(out=d["base"][:, ::2])):
        with pytest.raises(mb.MoeError):
            f(**bad)
    with pytest.raises(mb.MoeError, match="multiples of 8"):
        f(x=d["x"][:, :60].contiguous(), A=d["A"][:, :, :60].contiguous())
    with pytest.raises(mb.MoeError, match="rank"):
        z = torch.zeros(2, 129, 64, dtype=torch.bfloat16, device="cuda")
        f(A=z, B=torch.zeros(2, 129, 72, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(mb.MoeError, match="stride"):
        wide = torch.zeros(16, 80, dtype=torch.bfloat16, device="cuda")
        f(base=wide[:, :72], out=None, x=torch.zeros(16, 66, dtype=torch.bfloat16, device="cuda")[:, :64])


def test_infinite_sums_stay_infinite_at_odd_ranks():
    """Ranks that only pad r: 0 times infinity must not reach the row."""
    mb = _mb()
    d = _inputs(20, 64, 72, 2, 5, none=0.0)
    d["A"], d["B"] = d["A"].abs() + 0.125, d["B"].abs() + 0.125
    d["x"][3, 40] = float("inf")
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    torch.cuda.synchronize()
    assert torch.all(f["y"][3] == float("inf")) and torch.all(f["u"][3] == float("inf"))
    assert torch.isfinite(f["y"][[i for i in range(20) if i != 3]]).all()


@pytest.mark.parametrize("T", [90, 1500])
def test_other_adapters_gradients_do_not_see_an_infinite_row(T):
    mb = _mb()
    d = _inputs(T, 136, 264, 4, 24, none=0.1)
    ids = d["ids"][:, 0]
    rows = torch.nonzero(ids == 2)[:2, 0]
    run = lambda: mb.adapter_bwd(d["dy"], d["x"], u, d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])  # noqa: E731
    u = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"])["u"]
    ref = run()
    d["x"][rows[0]], d["dy"][rows[1]] = float("nan"), float("inf")
    got = run()
    torch.cuda.synchronize()
    keep = [0, 1, 3]
    assert torch.equal(got["dA"][keep], ref["dA"][keep]) and torch.equal(got["dB"][keep], ref["dB"][keep])
    other = torch.ones(T, dtype=torch.bool, device="cuda")
    other[rows[1]] = False
    assert torch.equal(got["dx"][other], ref["dx"][other])


def test_short_wait_limit_leaves_the_context_usable(set_option):
    """Waits that run out are reported in the status word; the same calls give the same results afterwards."""
    mb = _mb()
    d = _inputs(900, 1024, 520, 3, 64, seed=7)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def calls():
        f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"], status=status)
        g = mb.adapter_bwd(d["dy"], d["x"], u0, d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"], status=status)
        return f["y"], f["u"], g["dx"], g["dA"], g["dB"]

    u0 = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"])["u"]
    first = calls()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    set_option("WAIT_LIMIT_NS", 1)
    calls()
    torch.cuda.synchronize()
    assert int(status.item()) in (0, mb.STATUS_TIMEOUT)
    set_option("WAIT_LIMIT_NS", None)
    status.zero_()
    again = calls()
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("wide", ["H", "N"])
def test_past_32_bits(wide):
    """More than 2^31 numbers in x (or y and dy): the last rows, which are one adapter's, against 64 bits."""
    mb = _mb()
    T, n, r, tail = 530000, 3, 4, 100
    H, N = (4096, 64) if wide == "H" else (64, 4096)
    gen = torch.Generator(device="cuda").manual_seed(3)
    bf = torch.bfloat16
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=bf)  # noqa: E731
    x, dy = rand(T, H), rand(T, N)
    A, B = rand(n, r, H) * H ** -0.5, rand(n, r, N) * r ** -0.5
    ids = torch.randint(-1, 2, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    ids[-tail:] = 2
    meta = mb.route_meta(ids, n, 128)
    f = mb.adapter_fwd(x, A, B, meta)
    g = mb.adapter_bwd(dy, x, f["u"], A, B, meta)
    torch.cuda.synchronize()
    xt, dt, a, b = (np64(t) for t in (x[-tail:], dy[-tail:], A[2], B[2]))
    u, v = xt @ a.T, dt @ b.T
    eu, ev = _e(H) * (np.abs(xt) @ np.abs(a).T), _e(N) * (np.abs(dt) @ np.abs(b).T)
    assert np.all(np.abs(np64(f["u"][-tail:]) - u) <= eu)
    eu, ev = eu + HALF * (np.abs(u) + eu), ev + HALF * (np.abs(v) + ev)
    for got, ref, err, mag in ((f["y"][-tail:], u @ b, eu @ np.abs(b), np.abs(u) @ np.abs(b)),
                               (g["dx"][-tail:], v @ a, ev @ np.abs(a), np.abs(v) @ np.abs(a)),
                               (g["dA"][2], v.T @ xt, ev.T @ np.abs(xt), np.abs(v).T @ np.abs(xt)),
                               (g["dB"][2], u.T @ dt, eu.T @ np.abs(dt), np.abs(u).T @ np.abs(dt))):
        err = err + _e(tail + 8) * (mag + err)
        assert np.all(np.abs(np64(got) - ref) <= err + HALF * (np.abs(ref) + err))
    none = ids[:, 0] < 0
    assert torch.all(f["y"][none][-1000:] == 0) and torch.all(g["dx"][none][-1000:] == 0)


def test_status_refusals():
    mb = _mb()
    d = _inputs(16, 64, 72, 2, 8)
    u = torch.zeros(16, 8, device="cuda")
    for bad in (torch.zeros(1, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(mb.MoeError):
            mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], status=bad)
        with pytest.raises(mb.MoeError):
            mb.adapter_bwd(d["dy"], d["x"], u, d["A"], d["B"], d["meta"], status=bad)


@pytest.mark.parametrize("what", ["falling", "negative", "beyond", "all one", "indices", "none"])
def test_wrong_metadata_stays_inside(what):
    """Offsets that fall, leave [0, T] or never end, indices outside: wrong rows, but nothing beside the results is written."""
    mb = _mb()
    T, H, N, n, r = 150, 136, 264, 6, 20
    d = _inputs(T, H, N, n, r)
    off = d["meta"]["expert_offsets"].clone()
    idx, back = d["meta"]["x_gather_idx"].clone(), d["meta"]["s_reverse_scatter_idx"].clone()
    if what == "falling":
        off = off.flip(0).contiguous()
    elif what == "negative":
        off[1:4] = torch.tensor([-5, -2 ** 31, 40], dtype=torch.int32)
    elif what == "beyond":
        off[2:] = torch.tensor([10, 2 ** 31 - 1, 149, 3000, 2 ** 30], dtype=torch.int32)
    elif what == "all one":
        off[:] = torch.tensor([0, T, 0, T, 0, T, 0], dtype=torch.int32)
    elif what == "indices":
        idx[::3], idx[1::7], back[::5] = 2 ** 31 - 1, -2 ** 31, 10 ** 6
    else:
        off.zero_()
    meta = dict(expert_offsets=off, x_gather_idx=idx, s_reverse_scatter_idx=back)
    pad = 4096
    ybuf, xbuf = (torch.full((T * c + 2 * pad,), 7.0, dtype=torch.bfloat16, device="cuda") for c in (N, H))
    y, dx = ybuf[pad:-pad].view(T, N), xbuf[pad:-pad].view(T, H)
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], meta, scale=d["scale"], base=d["base"], out=y)
    mb.adapter_bwd(d["dy"], d["x"], torch.zeros_like(f["u"]), d["A"], d["B"], meta, scale=d["scale"], base=d["dbase"], out=dx)
    torch.cuda.synchronize()
    for b in (ybuf, xbuf):
        assert torch.all(b[:pad] == 7) and torch.all(b[-pad:] == 7)
    good = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    torch.cuda.synchronize()
    _check_fwd(d, good)


@pytest.mark.parametrize("T,n", [(1, 40), (3, 64), (17, 300), (40, 1024)])
def test_more_adapters_than_rows(T, n):
    mb = _mb()
    d = _inputs(T, 264, 136, n, 9, seed=T, none=0.1)
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])
    torch.cuda.synchronize()
    _check_fwd(d, f)
    _check_bwd(d, f["u"], g)


def test_uneven_adapters():
    """One adapter of most rows before hundreds of few: gradient ranges that hold many adapters and adapters in many ranges."""
    mb = _mb()
    T, n = 3000, 200
    d = _inputs(T, 136, 264, n, 20, seed=9, none=0.05, only=[0] * 150 + [7] * 40 + list(range(10, 200)))
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])
    torch.cuda.synchronize()
    _check_fwd(d, f)
    _check_bwd(d, f["u"], g)
