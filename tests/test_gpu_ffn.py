"""GPU parity of ffn_fwd / ffn_bwd against the float64 oracle: one token to many, sizes off the tiles, both activations and
column layouts, biases, strided rows, both tilings of the forward, accumulation, streams, graphs.

Bounds, elementwise.  u = 2^-24.  A product of K terms accumulated in fp32 in any order (truncating adds counted: 2 u) is off
by at most e(K) = 2 (K + 8) u times the sum of the terms' magnitudes.  The activation and its slope come from approximations
good to 2^-19 of their own scale (exp2 and reciprocal within 2 ulp, g log2(e) rounded: |g| u in the exponent, and SiLU', GELU'
are sums of terms at most (1 + |g|)).  |act'| <= 1.13.  Every rounding to bf16 is off by at most 2^-8 of the value."""
import numpy as np
import pytest
import torch

from helpers import np64, rel_fro
from oracle import ffn as of

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8
APX = 2.0 ** -19


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


def _e(K):
    return 2 * (K + 8) * U


def _inputs(T, H, I, bias, seed=0, strided=False):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    bf = torch.bfloat16
    d = dict(x=rand(T, H), W1=rand(H, 2 * I) * H ** -0.5, W2=rand(I, H) * I ** -0.5, dout=rand(T, H),
             b1=0.3 * rand(2 * I) if bias else None, b2=0.3 * rand(H) if bias else None)
    d = {k: None if v is None else v.to(bf).cuda() for k, v in d.items()}
    if strided:
        for k, pad in (("x", 24), ("dout", 8)):
            wide = torch.full((T, H + pad), float("nan"), dtype=bf, device="cuda")
            wide[:, :H] = d[k]
            d[k] = wide[:, :H]
    return d


def _check_fwd(d, got, gelu, il):
    x, W1, W2 = (np64(d[k]) for k in ("x", "W1", "W2"))
    b1, b2 = (None if d[k] is None else np64(d[k]) for k in ("b1", "b2"))
    out, h = of.forward(x, W1, W2, b1, b2, gelu, il)
    H, I = W1.shape[0], W2.shape[0]
    eh = _e(H + 1) * (np.abs(x) @ np.abs(W1) + (0 if b1 is None else np.abs(b1)))
    if got["h"] is not None:
        assert np.all(np.abs(np64(got["h"]) - h) <= eh + HALF * (np.abs(h) + eh))
    g, up = of.split(h, il)
    eg, eu = of.split(eh, il)
    act, _ = of.activation(g, gelu)
    ea = 1.13 * eg * (np.abs(up) + eu) + np.abs(act) * eu + APX * (1 + np.abs(g)) * np.abs(g * up)
    ea = ea + HALF * (np.abs(act * up) + ea)
    mag = (np.abs(act * up) + ea) @ np.abs(W2) + (0 if b2 is None else np.abs(b2))
    eo = ea @ np.abs(W2) + _e(I + 1) * mag
    assert np.all(np.abs(np64(got["out"]) - out) <= eo + HALF * (np.abs(out) + eo))
    # two independent roundings of at most 2^-8 / sqrt(3) each in the mean square
    assert rel_fro(np64(got["out"]), out) < 2 * HALF


def _check_bwd(d, h, got, gelu, il, bias, scale=1.0):
    x, W1, W2, dout = (np64(d[k]) for k in ("x", "W1", "W2", "dout"))
    hh = np64(h)
    T, H, I = x.shape[0], x.shape[1], W2.shape[0]
    ref = of.backward(dout, x, hh, W1, W2, gelu, il)
    g, up = of.split(hh, il)
    act, slope = of.activation(g, gelu)
    eda = _e(H) * (np.abs(dout) @ np.abs(W2).T)
    da = np.abs(ref["da"])
    edg = np.abs(up * slope) * eda + APX * (1 + np.abs(g)) ** 2 * np.abs(up) * (da + eda)
    edu = np.abs(act) * eda + APX * (1 + np.abs(g)) * np.abs(g) * (da + eda)
    raw = of.join(edg, edu, il)                                   # dh before its rounding
    edh = raw + HALF * (np.abs(ref["dh"]) + raw)
    ea = APX * (1 + np.abs(g)) * np.abs(g * up)
    ea = ea + HALF * (np.abs(ref["a"]) + ea)
    for n, A, eA, B in (("dx", np.abs(ref["dh"]), edh, np.abs(W1).T), ("dW1", None, None, None),
                        ("dW2", np.abs(ref["a"]).T, ea.T, np.abs(dout))):
        if n == "dW1":
            e = np.abs(x).T @ edh + _e(T) * (np.abs(x).T @ (np.abs(ref["dh"]) + edh))
        else:
            e = eA @ B + _e(2 * I if n == "dx" else T) * ((A + eA) @ B)
        r = ref[n] * scale
        if scale != 1:      # added twice in bf16: each product, and the sum
            e = e * 2 + HALF * np.abs(ref[n]) * 2
        assert np.all(np.abs(np64(got[n]) - r) <= e + HALF * (np.abs(r) + e)), n
        assert rel_fro(np64(got[n]), r) < 2 * HALF, n
    if bias:
        k = T * U * 2
        e1 = raw.sum(0) + k * (np.abs(ref["dh"]) + raw).sum(0)
        assert np.all(np.abs(np64(got["db1"]) - ref["db1"] * scale) <= scale * e1 + 4 * U * np.abs(ref["db1"]))
        assert np.all(np.abs(np64(got["db2"]) - ref["db2"] * scale) <= scale * k * np.abs(dout).sum(0) + 4 * U * np.abs(ref["db2"]))


CASES = [(1, 8, 8), (1, 512, 256), (5, 64, 72), (16, 128, 64), (17, 200, 40), (33, 256, 264), (127, 520, 128), (128, 64, 512),
         (129, 136, 200), (255, 72, 136), (256, 256, 128), (257, 264, 392), (700, 1000, 776)]
# (gelu, interleaved, bias)
HOWS = [(False, False, False), (False, True, True), (True, False, True), (True, True, False)]


@pytest.mark.parametrize("gelu,il,bias", HOWS)
@pytest.mark.parametrize("T,H,I", CASES)
@pytest.mark.parametrize("tiles", [1, 2])
def test_forward(T, H, I, gelu, il, bias, tiles, set_option):
    mb = _mb()
    set_option("FFN_TILES", tiles)
    d = _inputs(T, H, I, bias, seed=T + H, strided=(T + I) % 3 == 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mb.ffn_fwd(d["x"], d["W1"], d["W2"], d["b1"], d["b2"], glu=int(gelu), gate_up_layout=int(il), save=(T + H) % 2 == 0 or T < 9,
                     status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    _check_fwd(d, got, gelu, il)


@pytest.mark.parametrize("gelu,il,bias", HOWS)
@pytest.mark.parametrize("T,H,I", CASES)
def test_backward(T, H, I, gelu, il, bias):
    mb = _mb()
    d = _inputs(T, H, I, bias, seed=T + H, strided=(T + I) % 3 == 0)
    h = (d["x"].float() @ d["W1"].float() + (0 if d["b1"] is None else d["b1"].float())).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mb.ffn_bwd(d["dout"], d["x"], h, d["W1"], d["W2"], bias=bias, glu=int(gelu), gate_up_layout=int(il), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert (got["db1"] is not None) == bias
    _check_bwd(d, h, got, gelu, il, bias)


def test_many_tiles():
    """More tiles than CTA pairs in every kernel, with the tiling chosen by the library."""
    mb = _mb()
    T, H, I = 2900, 1032, 1160
    d = _inputs(T, H, I, True, seed=9)
    got = mb.ffn_fwd(d["x"], d["W1"], d["W2"], d["b1"], d["b2"], gate_up_layout=1)
    g = mb.ffn_bwd(d["dout"], d["x"], got["h"], d["W1"], d["W2"], bias=True, gate_up_layout=1)
    torch.cuda.synchronize()
    _check_fwd(d, got, False, True)
    _check_bwd(d, got["h"], g, False, True, True)


def test_accumulate_and_repeat():
    mb = _mb()
    d = _inputs(300, 136, 200, True, seed=3)
    h = mb.ffn_fwd(d["x"], d["W1"], d["W2"], d["b1"], d["b2"])["h"]
    call = lambda **k: mb.ffn_bwd(d["dout"], d["x"], h, d["W1"], d["W2"], bias=True, **k)  # noqa: E731
    a, b = call(), call()
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]), k
    c = call(accumulate_into=b)
    torch.cuda.synchronize()
    assert c["dW1"] is b["dW1"] and torch.equal(c["dx"], a["dx"])
    for k in ("dW1", "dW2"):        # x + x is exact in bf16
        assert torch.equal(c[k], 2 * a[k]), k
    for k in ("db1", "db2"):
        assert torch.equal(c[k], 2 * a[k]), k


def test_rows_do_not_depend_on_the_batch():
    """A token's output is the same bit for bit whatever other tokens the batch holds, within one token tile."""
    mb = _mb()
    d = _inputs(12, 256, 128, True, seed=4)
    full = mb.ffn_fwd(d["x"], d["W1"], d["W2"], d["b1"], d["b2"])
    one = mb.ffn_fwd(d["x"][7:8], d["W1"], d["W2"], d["b1"], d["b2"])
    torch.cuda.synchronize()
    assert torch.equal(full["out"][7:8], one["out"]) and torch.equal(full["h"][7:8], one["h"])


def test_no_rows():
    mb = _mb()
    d = _inputs(3, 64, 32, True)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    r = mb.ffn_fwd(e, d["W1"], d["W2"])
    assert r["out"].shape == (0, 64) and r["h"].shape == (0, 64)
    g = mb.ffn_bwd(e, e, r["h"], d["W1"], d["W2"], bias=True)
    torch.cuda.synchronize()
    assert all(torch.all(g[k] == 0) for k in ("dW1", "dW2", "db1", "db2")) and g["dx"].shape == (0, 64)
    g["dW1"].fill_(3)
    g2 = mb.ffn_bwd(e, e, r["h"], d["W1"], d["W2"], bias=True, accumulate_into=g)
    torch.cuda.synchronize()
    assert torch.all(g2["dW1"] == 3)


def test_rows_behind_the_last_are_left_alone():
    """Tiles reach past the last row and column; nothing there is written, and what lies there (NaN) is not read."""
    mb = _mb()
    T, H, I = 131, 72, 40
    lib = mb.lib()
    d = _inputs(T, H, I, True, seed=5)
    bf = torch.bfloat16
    wide = torch.full((T + 200, H), float("nan"), dtype=bf, device="cuda")
    wide[:T] = d["x"]
    for tiles in (1, 2):
        with mb.option("FFN_TILES", tiles):
            out = torch.full((T + 200, H), 7.0, dtype=bf, device="cuda")
            h = torch.full((T + 200, 2 * I), 7.0, dtype=bf, device="cuda")
            ws = torch.empty(lib.ffn_fwd_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")
            st = torch.cuda.current_stream().cuda_stream
            p = lambda t: t.data_ptr()  # noqa: E731
            assert lib.ffn_fwd(p(wide), H, p(d["W1"]), p(d["b1"]), p(d["W2"]), p(d["b2"]), T, H, I, 0, 0, p(h), p(out), None, p(ws),
                               ws.numel(), st) == 0
            torch.cuda.synchronize()
            assert torch.all(out[T:] == 7) and torch.all(h[T:] == 7)
            _check_fwd(d, dict(out=out[:T], h=h[:T]), False, False)


def test_extreme_values():
    """Gates far out keep their limits (SiLU and GELU are 0 or g there), infinities and NaN stay in their own rows."""
    mb = _mb()
    H = I = 64
    T = 40
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.linspace(-300, 300, T)
    W1 = torch.zeros(H, 2 * I, dtype=torch.bfloat16, device="cuda")
    W1[0, :I], W1[1, I:] = 1, 1
    x[:, 1] = 1
    W2 = torch.eye(I, H, dtype=torch.bfloat16, device="cuda")
    x[11, 5] = float("nan")
    x[12, 5] = float("inf")
    for gelu in (0, 1):
        for tiles in (1, 2):
            with mb.option("FFN_TILES", tiles):
                r = mb.ffn_fwd(x, W1, W2, glu=gelu)
                torch.cuda.synchronize()
            keep = [i for i in range(T) if i not in (11, 12)]
            ref = of.activation(np64(x[keep, :1]), bool(gelu))[0]
            assert np.all(np.abs(np64(r["out"][keep]) - ref) <= 3 * HALF * np.abs(ref) + 1e-6)
            assert torch.all(torch.isnan(r["out"][11])) and torch.all(torch.isnan(r["out"][12]))


def test_streams_and_graph():
    mb = _mb()
    d = _inputs(150, 136, 72, True, seed=6)

    def calls(stream=None):
        f = mb.ffn_fwd(d["x"], d["W1"], d["W2"], d["b1"], d["b2"], stream=stream)
        g = mb.ffn_bwd(d["dout"], d["x"], f["h"], d["W1"], d["W2"], bias=True, stream=stream)
        return [f["out"], f["h"]] + [g[k] for k in ("dx", "dW1", "dW2", "db1", "db2")]

    ref = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        h1 = calls()
    with torch.cuda.graph(g2):
        h2 = calls()
    d["x"].mul_(-0.5)
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    now = calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(now, h1, h2))


def test_refusals():
    mb = _mb()
    d = _inputs(4, 64, 32, True)
    f = lambda **k: mb.ffn_fwd(**{**dict(x=d["x"], W1=d["W1"], W2=d["W2"], b1=d["b1"], b2=d["b2"]), **k})  # noqa: E731
    for bad in (dict(x=d["x"].cpu()), dict(x=d["x"].float()), dict(x=d["x"][:, ::2]), dict(W1=d["W1"][:, :-2]), dict(W2=d["W2"].t()),
                dict(b1=d["b1"].float()), dict(b2=d["b2"][:-8]), dict(glu=2), dict(gate_up_layout=2),
                dict(status=torch.zeros(1, device="cuda"))):
        with pytest.raises(mb.MoeError):
            f(**bad)
    wide = torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mb.MoeError, match="row stride"):
        f(x=wide[:, :64])
    with pytest.raises(mb.MoeError, match="aligned"):
        f(x=torch.zeros(4, 72, dtype=torch.bfloat16, device="cuda")[:, 4:68])
    with pytest.raises(mb.MoeError, match="multiples of 8"):
        mb.ffn_fwd(wide[:, :60].contiguous(), torch.zeros(60, 64, dtype=torch.bfloat16, device="cuda"),
                   torch.zeros(32, 60, dtype=torch.bfloat16, device="cuda"))
