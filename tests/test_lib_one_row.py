"""CPU checks of the entry points' row strides: with one row there is no next one, so any stride passes; with two rows a stride
below the width or off 8 elements is refused, before any launch."""
import pytest

INVALID = -1
A = 1 << 20          # an aligned address that a refused call never reads


@pytest.fixture(scope="module")
def lib():
    from moe_expert_layer_routing_gb300 import _build
    _build.build()
    import moe_expert_layer_routing_gb300 as mb
    return mb.lib()


def _ffn_fwd(lib, T, ld):
    return lib.ffn_fwd(A, ld, A, None, A, None, T, 64, 32, 0, 0, None, A, None, A + 16, 1 << 30, None)


def _ffn_bwd_x(lib, T, ld):
    return lib.ffn_bwd(A, 64, A, ld, A, A, A, T, 64, 32, 0, 0, A, A, A, None, None, 0, None, A + 16, 1 << 30, None)


def _ffn_bwd_dout(lib, T, ld):
    return lib.ffn_bwd(A, ld, A, 64, A, A, A, T, 64, 32, 0, 0, A, A, A, None, None, 0, None, A + 16, 1 << 30, None)


def _adapter_fwd(lib, T, x=64, base=72, out=A + 4096):
    return lib.adapter_fwd(A, x, A, A, None, A, base, A, A, A, T, 64, 72, 2, 4, out, None, None, A + 16, 1 << 30, None)


def _adapter_bwd(lib, T, dy=72, x=64, base=64, out=A + 4096):
    return lib.adapter_bwd(A, dy, A, x, A, A, A, None, A, base, A, A, A, T, 64, 72, 2, 4, out, A, A, 0, None, A + 16, 1 << 30, None)


CALLS = {"ffn_fwd x": _ffn_fwd, "ffn_bwd x": _ffn_bwd_x, "ffn_bwd dout": _ffn_bwd_dout,
         "adapter_fwd x": lambda lib, T, ld: _adapter_fwd(lib, T, x=ld),
         "adapter_fwd base": lambda lib, T, ld: _adapter_fwd(lib, T, base=ld),
         "adapter_fwd base in place": lambda lib, T, ld: _adapter_fwd(lib, T, base=ld, out=A),
         "adapter_bwd dy": lambda lib, T, ld: _adapter_bwd(lib, T, dy=ld),
         "adapter_bwd x": lambda lib, T, ld: _adapter_bwd(lib, T, x=ld),
         "adapter_bwd base": lambda lib, T, ld: _adapter_bwd(lib, T, base=ld),
         "adapter_bwd base in place": lambda lib, T, ld: _adapter_bwd(lib, T, base=ld, out=A)}


@pytest.mark.parametrize("ld", [1, 68, 216, 1 << 40])
@pytest.mark.parametrize("name", CALLS)
def test_one_row(lib, name, ld):
    """The call passes the strides and is refused for its workspace's alignment, which is asked last."""
    assert CALLS[name](lib, 1, ld) == INVALID
    assert b"256-byte" in lib.moe_last_error()


@pytest.mark.parametrize("ld", [1, 68])
@pytest.mark.parametrize("name", CALLS)
def test_two_rows(lib, name, ld):
    assert CALLS[name](lib, 2, ld) == INVALID
    assert b"stride" in lib.moe_last_error()
