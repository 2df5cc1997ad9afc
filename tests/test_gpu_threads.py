"""The library called from several host threads at once."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

_THREADS = r"""
import threading, torch
import moe_expert_layer_routing_gb300 as mb
widths = [2056 + 8 * i for i in range(32)] + [2049 + 32 * i for i in range(32)]
x = {H: torch.randn(5, H, generator=torch.Generator("cuda").manual_seed(H), device="cuda") for H in widths}
one = torch.ones(8192, device="cuda")
torch.cuda.synchronize()
mb.lib()
gate, got, wrong = threading.Barrier(16), {}, []
def work(k):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            gate.wait()
            for H in widths[k::16][::1 if k % 2 else -1]:
                f = mb.layer_norm_fwd(x[H], one[:H])
                b = mb.layer_norm_bwd(x[H], x[H], one[:H], f["mean"], f["rstd"])
                got[H] = [f["y"], b["dx"], b["dgamma"]]
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        wrong.append(repr(e))
threads = [threading.Thread(target=work, args=(k,)) for k in range(16)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not wrong, wrong
for H in widths:
    f = mb.layer_norm_fwd(x[H], one[:H])
    b = mb.layer_norm_bwd(x[H], x[H], one[:H], f["mean"], f["rstd"])
    assert all(torch.equal(p, q) for p, q in zip(got[H], [f["y"], b["dx"], b["dgamma"]])), H
print("same")
"""


def test_first_calls_from_many_threads():
    """In a new process sixteen threads make the first calls of the same kernels with different shared-memory sizes: every
    launch gets what it needs, and the results are those of calls one after another."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _THREADS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
