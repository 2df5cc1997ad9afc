"""The example's training step (layer norm, router with its losses, 8-bit checkpoint, moe_bwd, their backward passes
chained) against float64 automatic differentiation of the whole block."""
import importlib.util
import os

import pytest
import torch

from helpers import BF16_TOL, np64, rel_fro

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _inputs(T, H):
    gen = torch.Generator(device="cuda").manual_seed(3)
    return [torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3)]


def test_gradients_of_the_chained_step():
    """Every gradient of <dout, out> + balance + z.  The reference takes the values the step stores in fewer bits (y in
    bf16, gate and up in 8 bits) as they are and differentiates past the rounding; what remains is bf16 rounding in
    moe_bwd and of its inputs, the bar of that path."""
    ex = _example()
    mb = ex.mb
    T, H, I, E, K = 300, 128, 128, 8, 2
    blk = ex.Block(H, I, E, K, alpha=0.5, beta=0.05)
    x, r, dout = _inputs(T, H)
    seg = torch.tensor([0, 100, 100, 290], dtype=torch.int32, device="cuda")
    out, aux, saved = blk.forward(x, r, seg)
    dout[290:] = 0          # padding tokens take no part
    got = blk.backward(dout, saved)
    torch.cuda.synchronize()
    assert int(got["status"].item()) == 0 and int(saved["route"]["status"].item()) == 0
    stream = saved["norm"]["sum"].double().requires_grad_()
    p = {k: getattr(blk, k).double().requires_grad_() for k in ("gamma", "beta_norm", "Wr", "W1", "W2")}
    y = torch.nn.functional.layer_norm(stream, (H,), p["gamma"], p["beta_norm"], ex.EPS)
    y = saved["norm"]["y"].double() + (y - y.detach())
    logits = y @ p["Wr"]
    prob = torch.softmax(logits, -1)
    ids = saved["route"]["ids"].long()
    assert torch.equal(ids[:290].sort(-1)[0], torch.topk(logits[:290], K, -1)[1].sort(-1)[0]) and torch.all(ids[290:] == -1)
    sel = torch.gather(prob, 1, ids.clamp(min=0))
    s = sel / sel.sum(-1, keepdim=True)
    meta = mb.route_meta(saved["route"]["ids"], E, blk.B)
    ends = meta["expert_offsets"].tolist()
    h8 = mb.ckpt8_unpack(saved["ckpt_q"], saved["ckpt_sf"], meta, ends[-1]).double()
    total = (stream * dout.double()).sum()
    for e in range(E):
        rows = slice(ends[e], ends[e + 1])
        t, flat = meta["x_gather_idx"][rows].long(), meta["s_scatter_idx"][rows].long()
        xw = y[t] @ p["W1"][e]
        h = h8[rows] + (xw - xw.detach())
        a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        total = total + (s.flatten()[flat][:, None] * (a @ p["W2"][e]) * dout.double()[t]).sum()
    loss = torch.zeros((), dtype=torch.float64, device="cuda")
    for i, (lo, hi) in enumerate(((0, 100), (100, 100), (100, 290))):
        if hi > lo:
            c = saved["route"]["counts"][i].double()
            loss = loss + blk.alpha * (hi - lo) / 290 * (E * c / (K * (hi - lo)) * prob[lo:hi].mean(0)).sum()
    z = blk.beta / 290 * torch.logsumexp(logits[:290], -1).square().sum()
    assert abs(loss.item() - aux[0].item()) < 1e-5 * loss.item() and abs(z.item() - aux[1].item()) < 1e-5 * z.item()
    (total + loss + z).backward()
    ref = dict(stream=stream.grad, gamma=p["gamma"].grad, beta=p["beta_norm"].grad, Wr=p["Wr"].grad, W1=p["W1"].grad,
               W2=p["W2"].grad)
    errs = {k: rel_fro(np64(got[k]), np64(v)) for k, v in ref.items()}
    assert all(e < BF16_TOL for e in errs.values()), errs


def test_backward_repeats_bit_for_bit():
    """Every reduction of the chained backward has a fixed order."""
    ex = _example()
    blk = ex.Block(128, 128, 8, 2)
    x, r, dout = _inputs(512, 128)
    seg = torch.tensor([0, 200, 512], dtype=torch.int32, device="cuda")
    _, _, saved = blk.forward(x, r, seg)
    a, b = blk.backward(dout, saved), blk.backward(dout, saved)
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_calls_captured_into_a_graph_replay_to_the_eager_results():
    """Layer norm, router with its losses, their gradients, activation and read-back captured once; the replay reads the
    inputs as they then are."""
    ex = _example()
    mb = ex.mb
    T, H, E, K, I, B = 200, 320, 24, 3, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, dy, logits = rand(T, H).to(torch.bfloat16), rand(T, H).to(torch.bfloat16), rand(T, E)
    h = rand(T * K, 2 * I).to(torch.bfloat16)
    gamma = torch.ones(H, device="cuda")
    seg = torch.tensor([0, 90, 200], dtype=torch.int32, device="cuda")
    meta = mb.route_meta(mb.router_fwd(0, logits, K)["ids"], E, B)

    def calls():
        n = mb.layer_norm_fwd(x, gamma, gamma)
        b = mb.layer_norm_bwd(dy, x, gamma, n["mean"], n["rstd"])
        r = mb.router_fwd(0, logits, K, seg_offsets=seg, alpha=0.1, beta=0.1)
        d = mb.balance_bwd(logits, r["lse"], r["counts"], K, seg_offsets=seg, alpha=0.1, beta=0.1)
        g = mb.glu_fwd(h, meta, B)
        u = mb.ckpt8_unpack(g["ckpt_q"], g["ckpt_sf"], meta, T * K)
        return [n["y"], b["dx"], b["dgamma"], b["dbeta"], r["ids"], r["scores"], r["loss"], r["counts"], d, g["a"], u]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for t in (x, dy, logits, h):
        t.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, calls()):
        assert torch.equal(a, b)
