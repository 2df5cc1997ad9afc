"""scale u and v enter the adapters' second products as two bf16 numbers each, together off by at most 2^-16: shown where the
result's own rounding does not hide it, on sums that a base (or an earlier result) cancels to what its rounding left.

Bounds, elementwise, as in the parity tests: u = 2^-24, a sum of K products in fp32 is off by at most e(K) = 2 (K + 8) u times
the sum of the terms' magnitudes (truncating adds counted), a rounding to bf16 by at most 2^-8 of the value.  The two parts have
one sign, so the terms' magnitudes are those of one operand (to 2^-16 of them, which the 8 in e(K) more than covers), in twice
as many terms.  Where the first sums are short enough (up to 136 terms) for their own bound not to hide it, each test also asks
that a single bf16 operand, truncated or rounded, would break the bound."""
import numpy as np
import pytest
import torch

from helpers import np64

pytestmark = pytest.mark.gpu
U, HALF, PAIR = 2.0 ** -24, 2.0 ** -8, 2.0 ** -16


def _e(K):
    return 2 * (K + 8) * U


def _bf16(v):
    return torch.from_numpy(v).float().to(torch.bfloat16)


def _singles(v):
    """v as one bf16 number: rounded, and truncated."""
    t = torch.from_numpy(np.ascontiguousarray(v)).float()
    return np64(t.to(torch.bfloat16)), np64((t.view(torch.int32) & -65536).view(torch.float32))


def _within(got, ref, bound, singles, short):
    assert np.all(np.abs(np64(got) - ref) <= bound)
    for s in singles:
        assert not short or np.any(np.abs(s - ref) > bound)


@pytest.mark.parametrize("r", [1, 5, 16, 17, 32, 33, 64, 100, 128])
@pytest.mark.parametrize("T,H,N", [(9, 64, 72), (400, 72, 136), (150, 520, 392)])
def test_two_numbers_each(T, H, N, r):
    import moe_expert_layer_routing_gb300 as mb
    gen = torch.Generator().manual_seed(T + r)
    rand = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    n = 2
    x, dy, A, B = rand(T, H), rand(T, N), rand(n, r, H), rand(n, r, N)
    scale = torch.tensor([0.7, 1.9], device="cuda")
    ids = torch.arange(T, dtype=torch.int32)[:, None] % n
    meta = mb.route_meta(ids.cuda(), n, 128)
    xs, ds, As, Bs, c = (np64(t) for t in (x, dy, A, B, scale))
    rows = [np.flatnonzero(ids.numpy()[:, 0] == a) for a in range(n)]

    u = np.zeros((T, r))
    v = np.zeros((T, r))
    eu, ev = np.zeros_like(u), np.zeros_like(v)
    for a in range(n):
        u[rows[a]], eu[rows[a]] = xs[rows[a]] @ As[a].T, _e(H) * (np.abs(xs[rows[a]]) @ np.abs(As[a]).T)
        v[rows[a]], ev[rows[a]] = c[a] * (ds[rows[a]] @ Bs[a].T), c[a] * _e(N + 1) * (np.abs(ds[rows[a]]) @ np.abs(Bs[a]).T)

    def product(w, W):          # each row by its adapter's matrix
        out = np.zeros((T, W.shape[2]))
        for a in range(n):
            out[rows[a]] = w[rows[a]] @ W[a]
        return out

    cs = c[ids.numpy()[:, 0]][:, None]
    su, esu = cs * u, cs * eu
    esu = esu + (PAIR + 2 * U) * (np.abs(su) + esu)
    ev = ev + (PAIR + 2 * U) * (np.abs(v) + ev)

    # y and dx onto a base that leaves what its own rounding left
    base = _bf16(-product(su, Bs)).cuda()
    dbase = _bf16(-product(v, As)).cuda()
    f = mb.adapter_fwd(x, A, B, meta, scale=scale, base=base)
    g = mb.adapter_bwd(dy, x, f["u"], A, B, meta, scale=scale, base=dbase)
    torch.cuda.synchronize()
    for got, b, w, ew, W in ((f["y"], base, su, esu, Bs), (g["dx"], dbase, v, ev, As)):
        ref = np64(b) + product(w, W)
        e = product(ew, np.abs(W)) + _e(2 * r + 1) * (product(np.abs(w) + ew, np.abs(W)) + np.abs(np64(b)))
        _within(got, ref, e + HALF * (np.abs(ref) + e), [np64(b) + product(s, W) for s in _singles(w)], max(H, N) <= 136)

    # dA and dB onto an earlier result that does
    uu = np64(f["u"])
    sg = cs * uu                       # the backward's u is the forward's, in fp32
    esg = (PAIR + 2 * U) * np.abs(sg)

    def outer(w, rows_of):
        return np.stack([w[rows[a]].T @ rows_of[rows[a]] for a in range(n)])

    first = dict(dA=_bf16(-outer(v, xs)).cuda(), dB=_bf16(-outer(sg, ds)).cuda())
    old = {k: np64(t) for k, t in first.items()}
    mb.adapter_bwd(dy, x, f["u"], A, B, meta, scale=scale, base=dbase, accumulate_into=first)
    torch.cuda.synchronize()
    k = _e(2 * T + 8)
    for name, w, ew, m in (("dA", v, ev, xs), ("dB", sg, esg, ds)):
        ref = old[name] + outer(w, m)
        e = outer(ew, np.abs(m)) + k * (outer(np.abs(w) + ew, np.abs(m)) + np.abs(old[name]))
        _within(first[name], ref, e + HALF * (np.abs(ref) + e), [old[name] + outer(s, m) for s in _singles(w)], max(H, N) <= 136)
