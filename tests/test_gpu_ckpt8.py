"""The 8-bit gate/up checkpoint: glu_fwd's codes and scale bytes bit-exact against the oracle, its activation, the
values read back, and moe_bwd on the codes -- bit-identical to moe_bwd on a bf16 checkpoint holding the same values
(bf16 holds them exactly), in both precisions, layouts, activations and tile widths."""
import numpy as np
import pytest
import torch

from helpers import BF16_TOL, compare_outputs, np64
from moe_expert_layer_routing_gb300.inputs import (AFFINITY_ON_H, AFFINITY_ON_I, PREC_BF16, PREC_MXFP8, make_moe_inputs,
                                                   small_moe, with_ids)
from oracle import ckpt8 as oc
from oracle import moe as om
from oracle import route_meta as orm

pytestmark = pytest.mark.gpu


def _mb():
    import moe_expert_layer_routing_gb300 as mb
    return mb


def _ids(T, K, E, seed, unused=False):
    """Expert 0 empty, expert 1 one row, expert 2 hot."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(np.arange(2, E))[:K] for _ in range(T)])
    ids[: T // 2, 0] = 2
    for t in range(T // 2):
        if (ids[t, 1:] == 2).any():
            ids[t, 1 + int(np.argmax(ids[t, 1:] == 2))] = 2 + (np.setdiff1d(np.arange(2, E), ids[t])[0] - 2)
    ids[0, K - 1] = 1
    if unused:
        ids[3::5, K - 1] = -1
    return ids.astype(np.int32)


def _slots(meta, ids, E, B):
    """Block-layout slot of each grouped row, from the metadata tensors."""
    eo, bo = (meta[k].cpu().numpy().astype(np.int64) for k in ("expert_offsets", "block_offsets"))
    return np.concatenate([bo[e] * B + np.arange(eo[e + 1] - eo[e]) for e in range(E)])


@pytest.mark.parametrize("T,K,E,I,B", [(1, 1, 3, 64, 128), (37, 2, 5, 128, 128), (300, 3, 6, 64, 256), (200, 4, 9, 192, 512)])
@pytest.mark.parametrize("glu", [0, 1])
@pytest.mark.parametrize("interleaved", [0, 1])
def test_glu_fwd(T, K, E, I, B, glu, interleaved):
    mb = _mb()
    ids = _ids(T, K, E, T) if T > 1 else np.array([[2]], dtype=np.int32)
    if T == 200:
        ids[::4, K - 1] = -1
    meta = mb.route_meta(torch.from_numpy(ids).cuda(), E, B)
    R = T * K
    rng = np.random.default_rng(I)
    h = (rng.standard_normal((R, 2 * I)) * np.exp(2 * rng.standard_normal(2 * I))).astype(np.float32)
    h[:, 3] = 0.0
    h[:, 5] *= 2.0 ** -125
    h[:, 7] *= 2.0 ** 100
    h = torch.from_numpy(h).bfloat16()
    s = torch.rand(T, K, generator=torch.Generator().manual_seed(1))
    scaled = T % 2 == 1
    wide = torch.full((R, 2 * I + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, : 2 * I] = h.cuda()
    out = mb.glu_fwd(wide[:, : 2 * I] if scaled else h.cuda(), meta, B, glu=glu, gate_up_layout=interleaved,
                     s=s.cuda() if scaled else None)
    back = mb.ckpt8_unpack(out["ckpt_q"], out["ckpt_sf"], meta, R, gate_up_layout=interleaved)
    only = mb.glu_fwd(h.cuda(), meta, B, glu=glu, gate_up_layout=interleaved, checkpoint=False)
    torch.cuda.synchronize()
    valid = int(meta["expert_offsets"][-1])
    flat = meta["s_scatter_idx"].cpu().numpy()[:valid]
    hv = np64(h)[:valid]
    scale = s.double().numpy().reshape(-1)[flat] if scaled else None
    a = oc.activation(hv, "geglu" if glu else "swiglu", bool(interleaved), scale)
    # bf16 rounding 2^-8, and fp32's exp / erf and products: 2^-18 of |g u|
    g, u = (hv[:, 0::2], hv[:, 1::2]) if interleaved else (hv[:, :I], hv[:, I:])
    # a product that underflows fp32's range keeps an absolute error of 2^-126
    bound = 2.0 ** -8 * np.abs(a) + 2.0 ** -18 * np.abs(g * u) * (1 if scale is None else scale[:, None]) + 2.0 ** -126
    got = np64(out["a"])[:valid]
    big = np.abs(a) < 3e38
    assert np.all(np.abs(got - a)[big] <= bound[big])
    assert only["ckpt_q"] is None and (scaled or torch.equal(only["a"][:valid], out["a"][:valid]))
    # the checkpoint, slot by slot
    slot = _slots(meta, ids, E, B)
    N = meta["block_to_expert"].numel()
    cols = np.concatenate([np.arange(0, 2 * I, 2), np.arange(1, 2 * I, 2)]) if interleaved else np.arange(2 * I)
    dense = np.zeros((N * B, 2 * I))
    dense[slot] = hv[:, cols]
    q, sf = oc.pack(dense.reshape(N, B, 2, I).transpose(0, 2, 3, 1))
    tiles = np.unique(slot // 128)
    got_q = out["ckpt_q"].cpu().numpy().reshape(N, 2, I, B // 128, 128)
    got_sf = out["ckpt_sf"].cpu().numpy()
    for t in tiles:                                          # tiles without a row are not written
        n, b = divmod(int(t), B // 128)
        assert np.array_equal(got_q[n, :, :, b], q.reshape(N, 2, I, B // 128, 128)[n, :, :, b])
        assert np.array_equal(got_sf[n, :, b], sf[n, :, b])
    vals = oc.unpack(q, sf).transpose(0, 3, 1, 2).reshape(N * B, 2 * I)[slot]
    assert np.array_equal(np64(back)[:valid][:, cols], vals)


def test_groups_with_nan_and_infinity_read_as_nan():
    mb = _mb()
    T, E, I, B = 64, 2, 64, 128
    meta = mb.route_meta(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), E, B)
    h = torch.ones(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    h[5, 10], h[40, 70], h[41, 71] = float("nan"), float("inf"), float("-inf")
    out = mb.glu_fwd(h, meta, B)
    back = mb.ckpt8_unpack(out["ckpt_q"], out["ckpt_sf"], meta, T)
    bad = torch.zeros(T, 2 * I, dtype=torch.bool, device="cuda")
    bad[:32, 10] = bad[32:, 70] = bad[32:, 71] = True
    assert torch.equal(torch.isnan(back), bad) and torch.all(back[~bad] == 1)


def _problem(T, K, E, H, I, B, precision, affinity, bias=False, unused=False):
    cfg = small_moe(T=T, H=H, I=I, E=E, K=K, B=B, precision=precision, affinity=affinity, bias=bias, seed=11)
    inp = make_moe_inputs(cfg)
    return with_ids(inp, torch.from_numpy(_ids(T, K, E, 3, unused)))


def _grouped(inp, mb, interleaved):
    """Metadata and the grouped rows of the problem's checkpoint, and their 8-bit form."""
    cfg = inp.cfg
    meta = mb.route_meta(inp.ids.cuda(), cfg.E, cfg.block_size)
    slot = torch.from_numpy(_slots(meta, inp.ids.numpy(), cfg.E, cfg.block_size)).cuda()
    N, _, I, B = inp.ckpt.shape
    rows = inp.ckpt.cuda().permute(0, 3, 1, 2).reshape(N * B, 2, I)[slot]
    rows = (rows.transpose(1, 2) if interleaved else rows).reshape(-1, 2 * I).contiguous()
    c8 = mb.glu_fwd(rows, meta, B, gate_up_layout=interleaved)
    vals = mb.ckpt8_unpack(c8["ckpt_q"], c8["ckpt_sf"], meta, rows.shape[0], gate_up_layout=interleaved)
    vals = vals.reshape(-1, I, 2).transpose(1, 2) if interleaved else vals.reshape(-1, 2, I)
    ckpt = torch.zeros(N * B, 2, I, dtype=torch.bfloat16, device="cuda")
    ckpt[slot] = vals
    return c8, ckpt.reshape(N, B, 2, I).permute(0, 2, 3, 1).contiguous()


def _run(inp, mb, interleaved=0, glu=0, accumulate=False, **act):
    cfg = inp.cfg
    op = mb.MoeBwd(T=cfg.T, H=cfg.H, I=cfg.I, E=cfg.E, K=cfg.K, block_size=cfg.block_size, precision=cfg.precision,
                   affinity=cfg.affinity, has_bias=cfg.bias, glu=glu, gate_up_layout=interleaved, accumulate=accumulate,
                   act_src=mb.ACT_CHECKPOINT8 if "ckpt_q" in act else mb.ACT_CHECKPOINT)
    for t in (op.dW1, op.dW2):
        t.fill_(0.5)
    W1 = inp.W1.cuda()
    if interleaved:
        W1 = W1.reshape(cfg.E, cfg.H, 2, cfg.I).transpose(2, 3).reshape(cfg.E, cfg.H, 2 * cfg.I).contiguous()
    kw = dict(x=inp.x.cuda(), dout=inp.dout.cuda(), s=inp.s.cuda(), ids=inp.ids.cuda(), **act)
    if cfg.bias:
        kw["b2"] = inp.b2.cuda()
    if cfg.precision == PREC_MXFP8:
        (kw["W1_q"], kw["W1_sf"]), (kw["W2_q"], kw["W2_sf"]) = mb.quantize_weights(W1), mb.quantize_weights(inp.W2.cuda())
    else:
        kw.update(W1=W1, W2=inp.W2.cuda())
    op.bind(**kw).run()
    torch.cuda.synchronize()
    out = op.outputs()
    assert int(out["status"].item()) == 0
    return out


@pytest.mark.parametrize("T,K,E,H,I,B,precision,affinity,bias,glu,il,opts", [
    (200, 2, 6, 128, 256, 128, PREC_BF16, AFFINITY_ON_H, False, 0, 0, {}),
    (333, 3, 7, 256, 384, 256, PREC_BF16, AFFINITY_ON_I, True, 0, 0, {}),
    (150, 2, 5, 128, 256, 128, PREC_BF16, AFFINITY_ON_H, False, 1, 0, {}),
    (150, 2, 5, 128, 256, 512, PREC_BF16, AFFINITY_ON_I, False, 0, 1, {"MN_OPERANDS": 0}),
    (180, 2, 6, 128, 128, 1024, PREC_BF16, AFFINITY_ON_H, True, 0, 0, {"G1_GATHER": 1}),
    (260, 2, 6, 128, 384, 128, PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, {}),
    (260, 2, 6, 128, 256, 256, PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, {}),
    (260, 2, 6, 256, 384, 512, PREC_MXFP8, AFFINITY_ON_H, True, 1, 1, {}),
    (200, 2, 6, 128, 384, 128, PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, {"G1_TILE_N": 128, "G1_WARPS": 16}),
    (260, 2, 6, 128, 256, 256, PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, {"G1_TILE_N": 256}),
    (260, 2, 6, 128, 256, 128, PREC_BF16, AFFINITY_ON_H, False, 0, 0, {"G1_TILE_N": 128, "PDL": 0}),
])
def test_moe_bwd_on_codes_is_bit_identical_to_their_values_in_bf16(T, K, E, H, I, B, precision, affinity, bias, glu, il,
                                                                   opts, set_option):
    mb = _mb()
    for k, v in opts.items():
        set_option(k, v)
    inp = _problem(T, K, E, H, I, B, precision, affinity, bias, unused=T == 333)
    c8, ckpt = _grouped(inp, mb, il)
    # padding slots of a written tile hold zeros; no kernel may use what lies behind the rows
    got = _run(inp, mb, il, glu, accumulate=T == 150, ckpt_q=c8["ckpt_q"], ckpt_sf=c8["ckpt_sf"])
    ref = _run(inp, mb, il, glu, accumulate=T == 150, ckpt=ckpt)
    for k in ("dx", "dW1", "dW2", "ds", "db1", "db2"):
        if ref[k] is not None:
            if opts.get("G1_WARPS"):     # the bf16 run's sixteen warps add ds in another order
                compare_outputs({k: got[k]}, {k: np64(ref[k])}, 1e-6 if k == "ds" else 1e-12, names=(k,))
            else:
                assert torch.equal(got[k], ref[k]), k


def test_moe_bwd8_against_the_oracle():
    """The whole chain against float64: codes from the oracle's own packing of the checkpoint."""
    mb = _mb()
    inp = _problem(200, 2, 6, 128, 256, 128, PREC_BF16, AFFINITY_ON_H)
    cfg = inp.cfg
    q, sf = oc.pack(np64(inp.ckpt))
    got = _run(inp, mb, ckpt_q=torch.from_numpy(q).cuda(), ckpt_sf=torch.from_numpy(sf).cuda())
    meta = orm.route_meta(inp.ids.numpy(), cfg.E, cfg.block_size)
    h = orm.checkpoint_rows(oc.unpack(q, sf), meta, cfg.T, cfg.K)
    ref = om.moe_backward(inp.x, inp.dout, inp.W1, inp.W2, inp.s, inp.ids.numpy(), h)
    compare_outputs(got, ref, BF16_TOL)


def test_refusals():
    mb = _mb()
    meta = mb.route_meta(torch.zeros(8, 1, dtype=torch.int32, device="cuda"), 2, 128)
    h = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    N = meta["block_to_expert"].numel()
    q = torch.zeros(N, 2, 128, 128, dtype=torch.int8, device="cuda")
    sf = torch.zeros(mb.ckpt8_sf_shape(N, 128, 128), dtype=torch.uint8, device="cuda")
    for bad in (lambda: mb.glu_fwd(h[:, :96], meta, 128), lambda: mb.glu_fwd(h.float(), meta, 128),
                lambda: mb.glu_fwd(h, meta, 128, glu=2), lambda: mb.glu_fwd(h, meta, 128, gate_up_layout=2),
                lambda: mb.glu_fwd(h.cpu(), meta, 128), lambda: mb.ckpt8_unpack(q, sf.flatten(), meta, 8),
                lambda: mb.ckpt8_unpack(q[:, :1], sf, meta, 8)):
        with pytest.raises(mb.MoeError):
            bad()
    kw = dict(T=8, H=128, I=128, E=2, K=1, block_size=128)
    op = mb.MoeBwd(**kw, act_src=mb.ACT_CHECKPOINT8)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    common = dict(x=z(8, 128), dout=z(8, 128), s=torch.zeros(8, 1, device="cuda"),
                  ids=torch.zeros(8, 1, dtype=torch.int32, device="cuda"), W1=z(2, 128, 256), W2=z(2, 128, 128))
    with pytest.raises(mb.MoeError, match="8-bit checkpoint"):
        op.bind(**common, ckpt_q=q).run()
    with pytest.raises(mb.MoeError):
        mb.MoeBwd(**kw, act_src=3)


def test_status_word_of_the_caller():
    mb = _mb()
    kw = dict(T=8, H=128, I=128, E=2, K=1, block_size=128)
    for bad in (torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.uint8, device="cuda"),
                torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")):
        with pytest.raises(mb.MoeError, match="status"):
            mb.MoeBwd(**kw, status=bad)
    inp = _problem(200, 2, 6, 128, 256, 128, PREC_BF16, AFFINITY_ON_H)
    c8, _ = _grouped(inp, mb, 0)
    cfg = inp.cfg
    word = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    op = mb.MoeBwd(T=cfg.T, H=cfg.H, I=cfg.I, E=cfg.E, K=cfg.K, block_size=cfg.block_size, act_src=mb.ACT_CHECKPOINT8,
                   status=word)
    op.bind(x=inp.x.cuda(), dout=inp.dout.cuda(), s=inp.s.cuda(), ids=inp.ids.cuda(), W1=inp.W1.cuda(), W2=inp.W2.cuda(),
            ckpt_q=c8["ckpt_q"], ckpt_sf=c8["ckpt_sf"]).run()
    torch.cuda.synchronize()
    assert int(word.item()) == 0


def _padding(inp, mb):
    """[N, B]: slots of the block layout that no row has."""
    cfg = inp.cfg
    meta = mb.route_meta(inp.ids.cuda(), cfg.E, cfg.block_size)
    slot = torch.from_numpy(_slots(meta, inp.ids.numpy(), cfg.E, cfg.block_size)).cuda()
    N = meta["block_to_expert"].numel()
    free = torch.ones(N * cfg.block_size, dtype=torch.bool, device="cuda")
    free[slot] = False
    return free.reshape(N, cfg.block_size)


@pytest.mark.parametrize("precision,affinity,bias,glu,il,I,B,names,opts", [
    (PREC_BF16, AFFINITY_ON_H, False, 0, 0, 256, 128, ("gate_act_ckpt",), {}),
    (PREC_BF16, AFFINITY_ON_I, False, 1, 1, 384, 256, ("gate_act_ckpt", "intermediate_ckpt"), {}),
    (PREC_BF16, AFFINITY_ON_H, True, 0, 0, 256, 256, ("intermediate_ckpt", "down_proj_act_ckpt"), {}),
    (PREC_BF16, AFFINITY_ON_H, False, 0, 0, 256, 128, ("down_proj_act_ckpt", "gate_act_ckpt"), {"MN_OPERANDS": 0}),
    (PREC_BF16, AFFINITY_ON_I, False, 0, 0, 128, 512, ("scaled_intermediate_ckpt",), {}),
    (PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, 384, 128, ("gate_act_ckpt",), {}),
    (PREC_MXFP8, AFFINITY_ON_I, False, 1, 1, 256, 256, ("gate_act_ckpt", "scaled_intermediate_ckpt"), {}),
    (PREC_MXFP8, AFFINITY_ON_I, True, 0, 0, 256, 128, ("intermediate_ckpt",), {}),
    (PREC_MXFP8, AFFINITY_ON_H, False, 0, 0, 256, 256, ("intermediate_ckpt", "down_proj_act_ckpt"), {}),
])
def test_codes_with_saved_factors(precision, affinity, bias, glu, il, I, B, names, opts, set_option):
    """The forward's other saved values beside the codes, as beside a bf16 checkpoint of the codes' values: the same bits."""
    mb = _mb()
    for k, v in opts.items():
        set_option(k, v)
    inp = _problem(260, 2, 6, 128, I, B, precision, affinity, bias)
    c8, ckpt = _grouped(inp, mb, il)
    keep = ~_padding(inp, mb)
    gen = torch.Generator(device="cuda").manual_seed(5)
    saved = {}
    for n in names:
        if n == "down_proj_act_ckpt":
            v = torch.randn(keep.shape[0], B, inp.cfg.H, generator=gen, device="cuda") * keep[..., None]
        else:
            v = torch.randn(keep.shape[0], I, B, generator=gen, device="cuda") * keep[:, None]
        saved[n] = v.to(torch.bfloat16)
    got = _run(inp, mb, il, glu, ckpt_q=c8["ckpt_q"], ckpt_sf=c8["ckpt_sf"], **saved)
    ref = _run(inp, mb, il, glu, ckpt=ckpt, **saved)
    plain = _run(inp, mb, il, glu, ckpt_q=c8["ckpt_q"], ckpt_sf=c8["ckpt_sf"])
    for k in ("dx", "dW1", "dW2", "ds", "db1", "db2"):
        if ref[k] is not None:
            assert torch.isfinite(ref[k]).all() and torch.equal(got[k], ref[k]), k
    assert not torch.equal(got["dW2"], plain["dW2"])          # the saved values are what was used


@pytest.mark.parametrize("precision,affinity,bias,glu,il,I,B,gate_act,opts", [
    (PREC_BF16, AFFINITY_ON_H, False, 0, 0, 256, 128, False, {}),
    (PREC_BF16, AFFINITY_ON_I, True, 0, 0, 384, 256, False, {}),
    (PREC_BF16, AFFINITY_ON_H, True, 1, 0, 256, 128, False, {}),
    (PREC_BF16, AFFINITY_ON_H, False, 0, 1, 256, 512, False, {}),
    (PREC_BF16, AFFINITY_ON_H, False, 0, 0, 256, 128, True, {}),
    (PREC_BF16, AFFINITY_ON_H, True, 0, 0, 256, 256, False, {"MN_OPERANDS": 0}),
    (PREC_BF16, AFFINITY_ON_H, False, 0, 0, 256, 128, False, {"G1_GATHER": 1}),
    (PREC_BF16, AFFINITY_ON_H, False, 0, 0, 256, 128, False, {"G1_GATHER": 0}),
    (PREC_MXFP8, AFFINITY_ON_I, True, 0, 0, 384, 128, False, {}),
    (PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, 256, 256, False, {}),
    (PREC_MXFP8, AFFINITY_ON_H, False, 1, 1, 384, 512, False, {}),
    (PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, 256, 128, True, {}),
    (PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, 384, 128, False, {"G1_GATHER": 1}),
    (PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, 384, 128, False, {"G1_GATHER": 0}),
    (PREC_MXFP8, AFFINITY_ON_I, False, 0, 0, 256, 128, False, {"G1_WARPS": 16, "G1_TILE_N": 128}),
])
def test_what_lies_in_padding_slots_does_not_matter(precision, affinity, bias, glu, il, I, B, gate_act, opts, set_option):
    """NaN and infinities in a bf16 checkpoint's padding slots (a caller's uninitialised memory), any codes behind the last
    row and scale byte 255 (NaN) for groups without a row: the bits of the zero-padded run."""
    mb = _mb()
    for k, v in opts.items():
        set_option(k, v)
    inp = _problem(260, 2, 6, 128, I, B, precision, affinity, bias)
    c8, ckpt = _grouped(inp, mb, il)
    free = _padding(inp, mb)
    N = free.shape[0]
    gen = torch.Generator(device="cuda").manual_seed(6)
    junk = torch.randint(0, 3, ckpt.shape, generator=gen, device="cuda")
    junk = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda")[junk].to(torch.bfloat16)
    at = free[:, None, None, :].expand_as(ckpt)
    bad_ckpt = torch.where(at, junk, ckpt)
    codes = torch.randint(-128, 128, ckpt.shape, generator=gen, device="cuda").to(torch.int8)
    bad_q = torch.where(at, codes, c8["ckpt_q"])
    no_row = free.reshape(N, B // 128, 4, 32).all(-1)[:, None, :, None, :, None].expand_as(c8["ckpt_sf"])
    bad_sf = torch.where(no_row, torch.full_like(c8["ckpt_sf"], 255), c8["ckpt_sf"])
    saved, bad_saved = {}, {}
    if gate_act:
        v = torch.randn(N, I, B, generator=gen, device="cuda").to(torch.bfloat16)
        saved["gate_act_ckpt"] = torch.where(free[:, None], torch.zeros_like(v), v)
        bad_saved["gate_act_ckpt"] = torch.where(free[:, None], junk[:, 0], v)
    ref = _run(inp, mb, il, glu, ckpt=ckpt, **saved)
    got = _run(inp, mb, il, glu, ckpt=bad_ckpt, **bad_saved)
    got8 = _run(inp, mb, il, glu, ckpt_q=bad_q, ckpt_sf=bad_sf, **bad_saved)
    for k in ("dx", "dW1", "dW2", "ds", "db1", "db2"):
        if ref[k] is not None:
            assert torch.isfinite(ref[k]).all() and torch.equal(got[k], ref[k]), k
            if not opts.get("G1_WARPS"):      # (sixteen warps on the bf16 checkpoint alone: ds in another order)
                assert torch.equal(got8[k], ref[k]), k
            else:
                assert torch.isfinite(got8[k]).all(), k
