"""CPU checks of the layer norm, router / balance-loss and 8-bit checkpoint entry points: argument errors are found on
the host, in documented codes, before any launch; empty problems need no pointers; host-side sizes."""
import ctypes

import pytest

INVALID, UNSUPPORTED = -1, -2
A = 1 << 20          # an aligned address that a refused call never reads


@pytest.fixture(scope="module")
def lib():
    from moe_expert_layer_routing_gb300 import _build
    _build.build()
    import moe_expert_layer_routing_gb300 as mb
    return mb.lib()


@pytest.fixture(autouse=True)
def no_launches(lib):
    before = lib.moe_kernel_launches()
    yield
    assert lib.moe_kernel_launches() == before


def _ln_fwd(lib, kind=0, x=A, ldx=64, r=None, ldr=0, gamma=A, beta=A, dt=0, wt=1, T=4, H=64, eps=1e-5, y=A, s=None, mean=A,
            rstd=A):
    return lib.layer_norm_fwd(kind, x, ldx, r, ldr, gamma, beta, dt, wt, T, H, eps, y, s, mean, rstd, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(kind=2), INVALID, b"bad kind"), (dict(dt=2), INVALID, b"bad dtype"), (dict(wt=-1), INVALID, b"bad dtype"),
    (dict(H=0), INVALID, b"bad sizes"), (dict(T=-1), INVALID, b"bad sizes"), (dict(H=1 << 30, ldx=1 << 30), UNSUPPORTED, b"too large"),
    (dict(eps=-1.0), INVALID, b"eps"), (dict(eps=float("nan")), INVALID, b"eps"), (dict(x=None), INVALID, b"null"),
    (dict(rstd=None), INVALID, b"null"), (dict(mean=None), INVALID, b"mean"), (dict(r=A, ldr=64), INVALID, b"sum"),
    (dict(ldx=63), INVALID, b"row stride"), (dict(r=A, ldr=0, s=A), INVALID, b"row stride"), (dict(x=A + 1), INVALID, b"aligned"),
    (dict(gamma=A + 2), INVALID, b"aligned"), (dict(dt=1, y=A + 2), INVALID, b"aligned"),
])
def test_layer_norm_fwd(lib, kw, code, text):
    assert _ln_fwd(lib, **kw) == code
    assert text in lib.moe_last_error()


def test_layer_norm_empty_and_workspace(lib):
    assert _ln_fwd(lib, T=0, x=None, gamma=None, y=None, rstd=None, mean=None) == 0
    size = lib.layer_norm_bwd_workspace_size
    assert size(0, 64) == 0 and size(4, 0) == 0
    for T, H in ((1, 1), (7, 4096), (1 << 20, 8192), (1000, 20000)):
        assert size(T, H) >= 2 * 4 * H
    # bounded by what stays resident on the card, whatever the number of rows
    assert size(1 << 30, 4096) == size(1 << 20, 4096) <= 2 * 4 * 4096 * 304


def _ln_bwd(lib, kind=0, dy=A, lddy=64, x=A, ldx=64, gamma=A, mean=A, rstd=A, dres=None, ldres=0, dt=0, wt=1, T=4, H=64, dx=A,
            dg=A, db=A, acc=0, ws=A, nbytes=1 << 20):
    return lib.layer_norm_bwd(kind, dy, lddy, x, ldx, gamma, mean, rstd, dres, ldres, dt, wt, T, H, dx, dg, db, acc, ws, nbytes,
                              None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(kind=-1), INVALID, b"bad kind"), (dict(acc=2), INVALID, b"accumulate"), (dict(dg=None), INVALID, b"null"),
    (dict(dx=None), INVALID, b"null"), (dict(mean=None), INVALID, b"mean"), (dict(lddy=1), INVALID, b"row stride"),
    (dict(dres=A, ldres=5), INVALID, b"row stride"), (dict(dy=A + 1), INVALID, b"aligned"), (dict(ws=A + 128), INVALID, b"256-byte"),
    (dict(nbytes=8), INVALID, b"workspace too small"), (dict(ws=None), INVALID, b"null"),
])
def test_layer_norm_bwd(lib, kw, code, text):
    assert _ln_bwd(lib, **kw) == code
    assert text in lib.moe_last_error()


def _router(lib, mode=0, logits=A, ld=64, T=4, K=2, E=64, off=None, S=1, scores=A, ids=A, lse=A, counts=A, prob=A, loss=A,
            status=None, ws=A, nbytes=1 << 24):
    return lib.moe_router_fwd(mode, 0, logits, ld, T, K, E, off, S, 0.1, 0.1, scores, ids, lse, counts, prob, loss, status, ws,
                              nbytes, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(mode=3), INVALID, b"bad mode"), (dict(K=65, E=128, ld=128), UNSUPPORTED, b"K above 64"), (dict(K=65), INVALID, b"bad sizes"),
    (dict(K=0), INVALID, b"bad sizes"), (dict(E=1025, ld=1025), UNSUPPORTED, b"E above"), (dict(T=-1), INVALID, b"bad sizes"),
    (dict(S=0), INVALID, b"bad sizes"), (dict(S=2), INVALID, b"seg_offsets"), (dict(counts=None), INVALID, b"together"),
    (dict(T=(1 << 31) - 1), UNSUPPORTED, b"too many"), (dict(logits=None), INVALID, b"null"), (dict(scores=None), INVALID, b"null"),
    (dict(ld=63), INVALID, b"row stride"), (dict(ws=None), INVALID, b"null"), (dict(ws=A + 4), INVALID, b"256-byte"),
    (dict(nbytes=16), INVALID, b"workspace too small"), (dict(ids=A + 2), INVALID, b"4-byte"),
])
def test_router_fwd(lib, kw, code, text):
    assert _router(lib, **kw) == code
    assert text in lib.moe_last_error() and lib.moe_last_error().startswith(b"moe_router_fwd")


def test_balance_entry_points(lib):
    fwd = lambda **k: lib.moe_balance_fwd(k.get("logits", A), 64, k.get("ids", A), 4, 2, 64, k.get("off"), k.get("S", 1), 0.1,  # noqa: E731
                                          0.1, None, k.get("counts", A), A, A, None, A, 1 << 24, None)
    assert fwd(ids=None) == INVALID and b"null" in lib.moe_last_error()
    assert fwd(counts=None) == INVALID and b"together" in lib.moe_last_error()
    assert fwd(S=3) == INVALID and b"seg_offsets" in lib.moe_last_error()
    bwd = lambda **k: lib.moe_balance_bwd(k.get("logits", A), 64, k.get("lse", A), k.get("counts", A), k.get("T", 4), 2,  # noqa: E731
                                          k.get("E", 64), None, k.get("S", 1), 0.1, 0.1, None, k.get("add"), k.get("ld_add", 64),
                                          k.get("out", A), None, None)
    assert bwd(lse=None) == INVALID and bwd(counts=None) == INVALID and bwd(out=None) == INVALID
    assert bwd(S=2) == INVALID and bwd(E=1) == INVALID and bwd(add=A, ld_add=3) == INVALID and bwd(out=A + 1) == INVALID
    assert bwd(T=0, logits=None, lse=None, counts=None, out=None) == 0
    size = lib.moe_balance_workspace_size
    assert size(100, 2, 64, 4) > 0 and size(100, 2, 2000, 4) == 0 and size(100, 65, 64, 1) == 0


def _glu(lib, h=A, ldh=256, rows=4, I=128, E=2, B=128, N=3, glu=0, layout=0, eo=A, s=None, idx=None, a=A, q=A, sf=A):
    return lib.moe_glu_fwd(h, ldh, rows, I, E, B, N, glu, layout, eo, A, A, s, idx, 4, a, q, sf, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(I=96, ldh=192), UNSUPPORTED, b"multiple of 64"), (dict(B=100), UNSUPPORTED, b"block_size"), (dict(E=2000), UNSUPPORTED, b"E above"),
    (dict(rows=-1), INVALID, b"bad sizes"), (dict(glu=2), INVALID, b"bad glu"), (dict(layout=7), INVALID, b"gate_up_layout"),
    (dict(q=None), INVALID, b"together"), (dict(s=A), INVALID, b"together"), (dict(h=None), INVALID, b"null"),
    (dict(eo=None), INVALID, b"null"), (dict(ldh=255), INVALID, b"row stride"), (dict(ldh=260), INVALID, b"row stride"),
    (dict(a=A + 8), INVALID, b"16-byte"), (dict(N=1 << 40), UNSUPPORTED, b"too many"),
])
def test_glu_fwd(lib, kw, code, text):
    assert _glu(lib, **kw) == code
    assert text in lib.moe_last_error()


def test_ckpt8_unpack_and_empty(lib):
    un = lambda **k: lib.moe_ckpt8_unpack(k.get("q", A), A, k.get("rows", 4), k.get("I", 128), 2, k.get("B", 128), 3, 0, A, A, A,  # noqa: E731
                                          k.get("h", A), k.get("ldh", 256), None)
    assert un(q=None) == INVALID and un(h=A + 2) == INVALID and un(ldh=100) == INVALID
    assert un(I=100) == UNSUPPORTED and un(B=64) == UNSUPPORTED
    assert un(rows=0, q=None, h=None) == 0 and _glu(lib, rows=0, h=None, a=None) == 0


def test_moe_bwd_on_an_8_bit_checkpoint(lib):
    import moe_expert_layer_routing_gb300 as mb
    a = mb.MoeBwdArgs(T=256, H=128, I=256, E=4, K=2, block_size=128, act_src=mb.ACT_CHECKPOINT8)
    n8 = lib.moe_bwd_workspace_size(ctypes.byref(a))
    assert n8 > 0
    a.act_src = mb.ACT_CHECKPOINT
    assert lib.moe_bwd_workspace_size(ctypes.byref(a)) == n8      # the codes are read as they are
    a.act_src = 3
    assert lib.moe_bwd_workspace_size(ctypes.byref(a)) == 0 and b"act_src" in lib.moe_last_error()
    a.act_src = mb.ACT_CHECKPOINT8
    for f in ("x", "dout", "W1", "W2", "s", "ids", "dx", "dW1", "dW2", "ds", "status_dev"):
        setattr(a, f, A)
    a.workspace, a.workspace_bytes = A, 1 << 40
    assert lib.moe_bwd(ctypes.byref(a), None) == INVALID and b"8-bit checkpoint" in lib.moe_last_error()
    a.gate_up_ckpt_q, a.gate_up_ckpt_sf = A + 8, A
    assert lib.moe_bwd(ctypes.byref(a), None) == INVALID and b"16-byte" in lib.moe_last_error()


def test_python_layer_refuses_cpu_tensors(lib):
    import torch
    import moe_expert_layer_routing_gb300 as mb
    x, g = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(mb.MoeError):
        mb.layer_norm_fwd(x, g)
    with pytest.raises(mb.MoeError):
        mb.router_fwd(0, x, 2)
    with pytest.raises(mb.MoeError):
        mb.balance_bwd(x, torch.zeros(4), torch.zeros(1, 8, dtype=torch.int32), 2)


@pytest.mark.parametrize("kw", [dict(mean=A + 2), dict(rstd=A + 1)])
def test_layer_norm_statistics_alignment(lib, kw):
    for call, who in ((_ln_fwd, b"layer_norm_fwd"), (_ln_bwd, b"layer_norm_bwd")):
        assert call(lib, **kw) == INVALID
        assert who in lib.moe_last_error() and b"aligned" in lib.moe_last_error()


@pytest.mark.parametrize("kw", [dict(dg=A + 2), dict(db=A + 3)])
def test_layer_norm_weight_gradient_alignment(lib, kw):
    assert _ln_bwd(lib, **kw) == INVALID
    assert b"aligned" in lib.moe_last_error()


def test_checkpoint_blocks_past_32_bits(lib):
    assert _glu(lib, N=1 << 61) == UNSUPPORTED
    assert b"too many tiles" in lib.moe_last_error()


@pytest.mark.parametrize("K,E", [(2, 64), (1, 1), (8, 256), (64, 1024)])
@pytest.mark.parametrize("S", [1, 2, 1000])
def test_balance_workspace_of_an_empty_batch(lib, K, E, S):
    """T = 0 is a valid problem, and its workspace size is asked for like any other's."""
    size = lib.moe_balance_workspace_size
    assert 0 < size(0, K, E, S) <= size(1, K, E, S)


def test_moe_bwd_refuses_a_status_word_it_cannot_write(lib):
    """Before anything is allocated, so without a device too."""
    import torch
    import moe_expert_layer_routing_gb300 as mb
    kw = dict(T=8, H=128, I=128, E=2, K=1, block_size=128)
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32),
                torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(mb.MoeError, match="status must be a CUDA tensor of one int32"):
            mb.MoeBwd(**kw, status=bad)


@pytest.mark.parametrize("which", range(5))
def test_checkpoint_metadata_alignment(lib, which):
    """Offsets, block table, scores and their index that are not on a 4-byte boundary are refused on the host."""
    p = [A] * 5
    p[which] = A + 2
    assert lib.moe_glu_fwd(A, 256, 4, 128, 2, 128, 3, 0, 0, *p, 4, A, A, A, None) == INVALID
    assert b"moe_glu_fwd" in lib.moe_last_error() and b"4-byte" in lib.moe_last_error()
    if which < 3:
        assert lib.moe_ckpt8_unpack(A, A, 4, 128, 2, 128, 3, 0, *p[:3], A, 256, None) == INVALID
        assert b"moe_ckpt8_unpack" in lib.moe_last_error() and b"4-byte" in lib.moe_last_error()
