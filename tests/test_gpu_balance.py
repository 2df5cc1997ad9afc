"""GPU parity of router_fwd, balance_fwd and balance_bwd against the float64 oracle: ids and counts exactly, every
form of the scores, packed sequences (empty ones, boundaries off the chunks, padding tokens), masked experts and
rows with none left, ties, NaN and infinities, strides and widths of every kernel variant.

Bounds (u = 2^-24): exp is within 2 ulp + 2^-22 |argument| (ex2 of a product rounded once), so a probability is
off by at most (E + 8 + 4 R) u of itself, R the row's logit range; sums over T tokens add (T + 32) u."""
import numpy as np
import pytest
import torch

from helpers import np64
from oracle import balance as ob
from oracle import router as orr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
A, B = 0.3, 0.05


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


def _logits(T, E, seed, special=True):
    rng = np.random.default_rng(seed)
    lg = (2 * rng.standard_normal((T, E))).astype(np.float32)
    if special:
        lg[1::5, ::3] = lg[1::5, :1]          # equal values
        lg[2::7, : E // 2] = -np.inf          # masked experts
        lg[3::11] = -np.inf                   # none left
        lg[4::13] = np.round(lg[4::13])       # many ties, +0 and -0
    return lg


def _dev(lg, ld=None, shift=0):
    T, E = lg.shape
    ld = ld or E
    buf = torch.full((T * ld + shift,), float("nan"), device="cuda")
    out = buf[shift:shift + T * ld].view(T, ld)[:, :E]
    out.copy_(torch.from_numpy(lg))
    return out


def _seg(T, seed):
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(0, T + 1, 5))
    return [int(cuts[0])] + [int(cuts[1])] * 2 + [int(c) for c in cuts[2:]]     # padding in front and behind, one empty


def _t(seg):
    return None if seg is None else torch.tensor(seg, dtype=torch.int32, device="cuda")


def _tol(lg, n):
    finite = np.where(np.isfinite(lg), lg, 0.0)
    return (lg.shape[1] + n + 64 + 8 * np.abs(finite).max()) * U


SHAPES = [(1, 4, 4), (1, 1, 1), (33, 8, 2), (257, 64, 8), (100, 40, 3), (70, 128, 8), (65, 256, 8), (50, 130, 4), (41, 33, 8),
          (40, 256, 16), (37, 512, 9), (19, 132, 32), (9, 1024, 64), (11, 1023, 33), (8, 520, 5), (600, 16, 1), (30, 64, 64)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("mode,renorm", [(0, False), (1, False), (1, True), (2, False)])
def test_router_fwd(T, E, K, mode, renorm):
    mb = _mb()
    lg = _logits(T, E, T + E)
    seg = _seg(T, K) if T > 30 else None
    odd = (T + E + mode) % 3 == 0
    out = mb.router_fwd(mode, _dev(lg, E + 5 if odd else None, 1 if odd else 0), K, renorm=renorm, seg_offsets=_t(seg),
                        alpha=A, beta=B)
    torch.cuda.synchronize()
    ids = ob.topk(lg, K, seg)
    assert np.array_equal(out["ids"].cpu().numpy(), ids)
    assert int(out["status"].item()) == 0
    ref = ob.losses(lg, ids, A, B, seg)
    tol = _tol(lg, 0)
    assert np.all(np.abs(np64(out["scores"]) - ob.scores(mode, lg, ids, renorm)) <= tol * np.abs(ob.scores(mode, lg, ids, renorm)))
    lse, want = np64(out["lse"]), ref["lse"]
    assert np.array_equal(np.isfinite(lse), np.isfinite(want))
    fin = np.isfinite(want)
    assert np.all(np.abs(lse[fin] - want[fin]) <= tol * (1 + np.abs(want[fin])))
    assert np.array_equal(out["counts"].cpu().numpy(), ref["counts"])
    tolT = _tol(lg, T)
    assert np.all(np.abs(np64(out["prob_sum"]) - ref["prob_sum"]) <= tolT * ref["prob_sum"] + 1e-30)
    assert np.all(np.abs(np64(out["loss"]) - ref["loss"]) <= 2 * tolT * np.abs(ref["loss"]))


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("add", [False, True])
def test_balance_bwd(T, E, K, add):
    mb = _mb()
    lg = _logits(T, E, T + E)
    seg = _seg(T, K) if T > 30 else None
    ids = ob.topk(lg, K, seg)
    ref = ob.losses(lg, ids, A, B, seg)
    odd = (T + E + add) % 3 == 0
    base = np.random.default_rng(1).standard_normal((T, E)).astype(np.float32) if add else None
    dl = np.array([1.5, -0.5])
    got = np64(mb.balance_bwd(_dev(lg, E + 4 if odd else None), torch.from_numpy(ref["lse"]).float().cuda(),
                              torch.from_numpy(ref["counts"]).int().cuda(), K, seg_offsets=_t(seg), alpha=A, beta=B,
                              dloss=torch.from_numpy(dl).float().cuda(), add=_dev(base, E + 3 if odd else None) if add else None))
    want = ob.gradient(lg, ref["counts"], K, A, B, dl, seg, base)
    # the terms that cancel: p (c_j + sum c p) and lse p
    size = np.zeros((T, E))
    owner, S = ob._sequences(T, seg)
    n = max(1, int((owner >= 0).sum()))
    for t in range(T):
        if owner[t] >= 0 and np.isfinite(ref["lse"][t]):
            p = np.exp(lg[t].astype(np.float64) - ref["lse"][t])
            c = ref["counts"][owner[t]]
            size[t] = abs(dl[0]) * A * E / (K * n * (owner == owner[t]).sum()) * p * (c + (c * p).sum())
            size[t] += abs(dl[1]) * 2 * B / n * abs(ref["lse"][t]) * p
    assert np.all(np.abs(got - want) <= 2 * _tol(lg, 0) * size + U * np.abs(want) + 1e-30)


def test_balance_fwd_takes_other_ids():
    """ids of another selection: repeated, unused and out-of-range ids; padding tokens' ids are not read."""
    mb = _mb()
    T, E, K = 300, 24, 4
    lg = _logits(T, E, 9)
    seg = [10, 100, 260]
    ids = np.random.default_rng(2).integers(-1, E + 2, (T, K)).astype(np.int32)
    out = mb.balance_fwd(_dev(lg), torch.from_numpy(ids).cuda(), seg_offsets=_t(seg), alpha=A, beta=B)
    torch.cuda.synchronize()
    ref = ob.losses(lg, ids, A, B, seg)
    assert np.array_equal(out["counts"].cpu().numpy(), ref["counts"])
    assert np.all(np.abs(np64(out["loss"]) - ref["loss"]) <= 2 * _tol(lg, T) * np.abs(ref["loss"]))


def test_many_tokens_and_sequences():
    """More chunks than one pass of the grid, sequences of 0 to 3 tokens and of thousands; the sum over sequences is
    the whole batch's; twice gives the same bits."""
    mb = _mb()
    T, E, K = 70001, 32, 4
    lg = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    lens = np.concatenate([np.arange(900) % 4, [5000, 0, 20000, 1]])
    lens = np.concatenate([lens, [T - 7 - lens.sum()]])
    seg = np.concatenate([[0], np.cumsum(lens)]).tolist()
    one = mb.router_fwd(0, lg, K, alpha=A, beta=B, seg_offsets=_t([0, T - 7]))
    out = mb.router_fwd(0, lg, K, alpha=A, beta=B, seg_offsets=_t(seg))
    again = mb.router_fwd(0, lg, K, alpha=A, beta=B, seg_offsets=_t(seg))
    torch.cuda.synchronize()
    top = torch.topk(lg, K, dim=-1)[1].int()
    top[-7:] = -1
    assert torch.equal(out["ids"], top) and torch.equal(one["ids"], top)
    p = torch.softmax(lg.double(), -1)
    at = torch.tensor(seg, device="cuda")
    cum = torch.cat([torch.zeros(1, E, dtype=torch.float64, device="cuda"), p.cumsum(0)])
    want = cum[at[1:]] - cum[at[:-1]]
    assert torch.all((out["prob_sum"].double() - want).abs() <= 1e-5 * want + 1e-6)
    assert torch.equal(out["counts"].sum(0), one["counts"][0])
    assert torch.all(out["counts"].sum(1) == torch.from_numpy(lens * K).cuda())
    for k in out:
        assert torch.equal(out[k], again[k]), k
    n = T - 7
    bal = A * E / (K * n) * ((out["counts"].double() * want).sum(1) / torch.from_numpy(lens).cuda().clamp(min=1)).sum()
    assert abs(float(out["loss"][0]) - float(bal)) <= 1e-5 * float(bal)


def test_nan_and_infinite_logits():
    mb = _mb()
    lg = _logits(6, 16, 3, special=False)
    lg[1, 5] = np.nan
    lg[2, 3] = np.inf
    lg[3, [2, 9]] = -np.nan
    out = mb.router_fwd(0, _dev(lg), 3, alpha=A, beta=B)
    plain = mb.router_fwd(2, _dev(lg), 3, balance=False)
    torch.cuda.synchronize()
    ids = ob.topk(lg, 3)
    assert np.array_equal(out["ids"].cpu().numpy(), ids) and ids[1, 0] == 5 and ids[3, :2].tolist() == [2, 9]
    s = np64(out["scores"])
    assert np.isnan(s[[1, 2, 3]]).any(1).all() and np.isfinite(s[[0, 4, 5]]).all()
    assert np.isnan(np64(out["loss"])).all()
    assert np64(plain["scores"])[2, 0] == np.inf and set(plain) == {"scores", "ids", "lse"}


LOWEST = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("mask", [LOWEST, -1e9, -1e30])
def test_finite_masks_and_huge_logits(mask):
    """Experts masked with a large negative number instead of -inf, rows with nothing else (then uniform: the mask is a
    value like any other), and logits so large that neighbours differ by more than e^88 of each other."""
    mb = _mb()
    T, E, K = 60, 24, 4
    lg = _logits(T, E, 5, special=False)
    lg[::3, 5:] = mask
    lg[7] = mask
    lg[8] = np.arange(E, dtype=np.float32)[::-1] * 3e6
    lg[9] = 1e7 + np.arange(E, dtype=np.float32) * 3
    lg[10] = -1e7 + np.arange(E, dtype=np.float32)[::-1]
    out = mb.router_fwd(0, _dev(lg), K, alpha=A, beta=0.0)
    g = mb.balance_bwd(_dev(lg), out["lse"], out["counts"], K, alpha=A, beta=0.0)
    torch.cuda.synchronize()
    ids = ob.topk(lg, K)
    assert np.array_equal(out["ids"].cpu().numpy(), ids)
    s = ob.scores(0, lg, ids)
    tol = (E + 64 + 8 * 30) * U      # differences are exact or beyond e^-88 here: 30 covers the ordinary rows' range
    assert np.all(np.abs(np64(out["scores"]) - s) <= tol * s + 1e-37)
    ref = ob.losses(lg, ids, A, 0.0)
    assert np.all(np.abs(np64(out["prob_sum"]) - ref["prob_sum"]) <= (T * U + tol) * ref["prob_sum"] + 1e-37)
    assert abs(float(out["loss"][0]) - ref["loss"][0]) <= 2 * (T * U + tol) * ref["loss"][0] and float(out["loss"][1]) == 0.0
    want = ob.gradient(lg, ref["counts"], K, A, 0.0)
    lim = A * E / (K * T * T) * ref["counts"].max() * 2
    assert np.all(np.abs(np64(g) - want) <= 4 * tol * lim)


def test_bad_offsets_are_reported_and_stay_in_bounds():
    mb = _mb()
    T, E, K = 500, 16, 2
    lg = _dev(_logits(T, E, 4))
    for seg in ([0, 300, 200, T], [-5, T], [0, T + 9], [T, 0], [400, 100, 450, 2]):
        out = mb.router_fwd(0, lg, K, seg_offsets=_t(seg), alpha=A, beta=B)
        torch.cuda.synchronize()
        assert int(out["status"].item()) == mb.STATUS_BAD_SEGMENTS, seg
    good = mb.router_fwd(0, lg, K, seg_offsets=_t([0, T]), alpha=A, beta=B)
    assert int(good["status"].item()) == 0


def test_chain_with_router_bwd_matches_autograd():
    """router_fwd -> router_bwd -> balance_bwd(add=): the logits' gradient of <ds, s> + losses, against torch's
    float64 automatic differentiation of the same selection."""
    mb = _mb()
    T, E, K = 90, 32, 4
    lg = _logits(T, E, 7, special=False)
    seg = [0, 40, 85]
    x = _dev(lg)
    f = mb.router_fwd(1, x, K, renorm=True, seg_offsets=_t(seg), alpha=A, beta=B)
    ds = torch.randn(T, K, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) * 0.01
    ds[85:] = 0
    dr = mb.router_bwd(1, f["ids"], ds, E, logits=x.contiguous(), scores=f["scores"], renorm=True)
    got = np64(mb.balance_bwd(x, f["lse"], f["counts"], K, seg_offsets=_t(seg), alpha=A, beta=B, add=dr))
    l64 = torch.from_numpy(lg).double().requires_grad_()
    ids = f["ids"].cpu().long().clamp(min=0)
    p = torch.softmax(l64, -1)
    r = torch.gather(p, 1, ids)
    total = ((r / r.sum(-1, keepdim=True))[:85] * ds.cpu().double()[:85]).sum()
    for a, b in ((0, 40), (40, 85)):
        c = f["counts"].cpu().double()[0 if a == 0 else 1]
        total = total + A * (b - a) / 85 * (E * c / (K * (b - a)) * p[a:b].mean(0)).sum()
    total = total + B / 85 * torch.logsumexp(l64[:85], -1).square().sum()
    total.backward()
    ref = l64.grad.numpy()
    assert np.linalg.norm(got - ref) <= 3e-5 * np.linalg.norm(ref)       # the bar of the router backward


def test_empty_and_refusals():
    mb = _mb()
    out = mb.router_fwd(0, torch.empty(0, 8, device="cuda"), 2, alpha=A)
    torch.cuda.synchronize()
    assert not out["counts"].any() and not out["loss"].any() and out["ids"].shape == (0, 2)
    lg = torch.zeros(4, 8, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    lse, cnt = torch.zeros(4, device="cuda"), torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    for bad in (lambda: mb.router_fwd(3, lg, 2), lambda: mb.router_fwd(0, lg, 9), lambda: mb.router_fwd(0, lg, 0),
                lambda: mb.router_fwd(0, lg.double(), 2), lambda: mb.router_fwd(0, lg.cpu(), 2),
                lambda: mb.router_fwd(0, torch.zeros(2, 1100, device="cuda"), 2), lambda: mb.router_fwd(0, lg.t(), 2),
                lambda: mb.router_fwd(0, lg, 2, seg_offsets=torch.tensor([0, 4], device="cuda")),
                lambda: mb.balance_fwd(lg, ids.long()), lambda: mb.balance_bwd(lg, lse[:3], cnt, 2),
                lambda: mb.balance_bwd(lg, lse, cnt, 2, seg_offsets=_t([0, 2, 4])),
                lambda: mb.balance_bwd(lg, lse, cnt, 2, add=lg[:3])):
        with pytest.raises((mb.MoeError, RuntimeError)):
            bad()


@pytest.mark.parametrize("S", [31, 33, 1023, 1500, 40000])
def test_pieces_of_many_sequences(S):
    """Sequences of 0 to 2 tokens between padding at both ends; more of them than tokens."""
    mb = _mb()
    T, E, K = 1300, 16, 2
    rng = np.random.default_rng(S)
    lg = _logits(T, E, S)
    seg = np.sort(rng.integers(3, T - 4, S + 1)).astype(np.int64)
    ids = ob.topk(lg, K, seg.tolist())
    owner = np.searchsorted(seg, np.arange(T), side="right") - 1      # the last of the sequences that start there
    owner[np.arange(T) >= seg[-1]] = -1
    out = mb.router_fwd(0, _dev(lg), K, alpha=A, beta=B, seg_offsets=_t(seg.tolist()))
    assert np.array_equal(out["ids"].cpu().numpy(), ids) and int(out["status"].item()) == 0
    counts = np.zeros((S, E), np.int64)
    for t in np.flatnonzero(owner >= 0):
        for e in ids[t]:
            if e >= 0:
                counts[owner[t], e] += 1
    assert np.array_equal(out["counts"].cpu().numpy(), counts)
    got = np64(mb.balance_bwd(_dev(lg), out["lse"], out["counts"], K, seg_offsets=_t(seg.tolist()), alpha=A, beta=B))
    lse = np64(out["lse"])
    n, lens = int((owner >= 0).sum()), np.diff(seg)
    for t in range(T):
        if owner[t] < 0 or not np.isfinite(lse[t]):
            assert not got[t].any()
            continue
        p, c = np.exp(lg[t].astype(np.float64) - np.logaddexp.reduce(lg[t].astype(np.float64))), counts[owner[t]]
        bal, z = A * E / (K * n * lens[owner[t]]) * p, 2 * B / n * np.logaddexp.reduce(lg[t].astype(np.float64)) * p
        assert np.all(np.abs(got[t] - (bal * (c - (c * p).sum()) + z)) <= 2 * _tol(lg, 0) * (bal * (c + (c * p).sum()) + np.abs(z)) + 1e-30)


BAD_SEGMENTS = ([0, 300, 200, 500], [-5, 500], [0, 509], [500, 0], [400, 100, 450, 2])


def test_selection_without_losses_reports_bad_offsets():
    mb = _mb()
    lg = _dev(_logits(500, 16, 4))
    for seg in BAD_SEGMENTS:
        out = mb.router_fwd(0, lg, 2, seg_offsets=_t(seg), balance=False)
        assert int(out["status"].item()) == mb.STATUS_BAD_SEGMENTS, seg
    good = mb.router_fwd(0, lg, 2, seg_offsets=_t([0, 100, 500]), balance=False)
    assert int(good["status"].item()) == 0 and set(good) == {"scores", "ids", "lse", "status"}
    none = mb.router_fwd(0, torch.empty(0, 16, device="cuda"), 2, seg_offsets=_t([0, 0]), balance=False)
    assert int(none["status"].item()) == 0


def test_gradient_reports_bad_offsets():
    mb = _mb()
    T, E, K = 500, 16, 2
    lg = _dev(_logits(T, E, 4))
    f = mb.router_fwd(0, lg, K, alpha=A, beta=B)
    word = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    for seg in BAD_SEGMENTS:
        counts = torch.ones(len(seg) - 1, E, dtype=torch.int32, device="cuda")
        mb.balance_bwd(lg, f["lse"], counts, K, seg_offsets=_t(seg), alpha=A, beta=B, status=word)
        assert int(word.item()) == mb.STATUS_BAD_SEGMENTS, seg
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in (dict(), dict(seg_offsets=_t([0, T])), dict(stream=side)):
        word.fill_(77)
        torch.cuda.synchronize()
        d = mb.balance_bwd(lg, f["lse"], f["counts"], K, alpha=A, beta=B, status=word, **kw)
        torch.cuda.synchronize()
        assert int(word.item()) == 0 and torch.equal(d, mb.balance_bwd(lg, f["lse"], f["counts"], K, alpha=A, beta=B))
    for bad in (word.cpu(), word.float(), torch.zeros(2, dtype=torch.int32, device="cuda")):
        with pytest.raises(mb.MoeError, match="status"):
            mb.balance_bwd(lg, f["lse"], f["counts"], K, alpha=A, beta=B, status=bad)


@pytest.mark.parametrize("E", [24, 64, 200, 1000, 33])
@pytest.mark.parametrize("dl", [(float("inf"), 1.0), (1.0, float("-inf")), (float("nan"), float("nan"))])
def test_loss_gradients_that_are_not_finite_stay_out_of_padding(E, dl):
    """Padding tokens and tokens with every expert masked get `add` alone, or 0, whatever the losses' gradient is (an
    overflow of a scaled loss must not reach what takes no part)."""
    mb = _mb()
    T, K = 80, 3
    lg = _logits(T, E, 3, special=False)
    lg[20] = -np.inf
    seg = _t([10, 40, 40, 60])
    f = mb.router_fwd(0, _dev(lg), K, seg_offsets=seg, alpha=A, beta=B)
    base = torch.from_numpy(np.random.default_rng(1).standard_normal((T, E)).astype(np.float32)).cuda()
    out_of_it = torch.tensor([t < 10 or t >= 60 or t == 20 for t in range(T)], device="cuda")
    for add in (None, base):
        d = mb.balance_bwd(_dev(lg), f["lse"], f["counts"], K, seg_offsets=seg, alpha=A, beta=B, add=add,
                           dloss=torch.tensor(dl, device="cuda"))
        assert torch.equal(d[out_of_it], torch.zeros_like(d[out_of_it]) if add is None else add[out_of_it])
        assert not torch.isfinite(d[~out_of_it]).all()
