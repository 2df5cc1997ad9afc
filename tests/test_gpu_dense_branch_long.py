"""The adapters' and dropout's kernels where a CTA or a warp goes round its loop: more pieces of work than CTAs at the ranks
whose buffers are fewest, gradient ranges of many stages, rows of several segments of four steps with ragged ends.  Bounds are
those of the parity tests."""
import numpy as np
import pytest
import torch

from helpers import np64
from oracle import dropout as od
from test_gpu_adapter import _check_bwd, _check_fwd, _inputs
from test_gpu_dropout import OFFSET, SEED, _bound, _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("r", [16, 40, 64, 100, 128])
@pytest.mark.parametrize("T,H,N,n", [(9000, 1000, 1032, 3), (6000, 2056, 264, 40)])
def test_adapters(T, H, N, n, r):
    import moe_expert_layer_routing_gb300 as mb
    d = _inputs(T, H, N, n, r, seed=r, none=0.1)
    f = mb.adapter_fwd(d["x"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["base"])
    g = mb.adapter_bwd(d["dy"], d["x"], f["u"], d["A"], d["B"], d["meta"], scale=d["scale"], base=d["dbase"])
    torch.cuda.synchronize()
    _check_fwd(d, f)
    _check_bwd(d, f["u"], g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(5000, 1160), (5000, 2048), (9100, 1032), (20000, 264)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("pad", [0, 16])
def test_dropout(dtype, T, H, residual, pad):
    import moe_expert_layer_routing_gb300 as mb
    p = 0.2
    x = _rand(T, H, dtype, 1, H + pad)
    r = _rand(T, H, dtype, 2, H + pad) if residual else None
    y = mb.dropout_fwd(x, p, SEED, OFFSET, residual=r)
    torch.cuda.synchronize()
    xs, rs = np64(x), None if r is None else np64(r)
    ref = od.forward(xs, p, SEED, OFFSET, rs)
    assert np.all(np.abs(np64(y) - ref) <= _bound(xs, rs, p, dtype, ref))
    if r is None:
        assert np.array_equal(np64(y) != 0, od.keep(T, H, p, SEED, OFFSET))
        assert torch.equal(mb.dropout_bwd(x, p, SEED, OFFSET), y)
