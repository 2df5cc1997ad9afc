"""Python binding of libmoebwd: MoE expert-layer backward (BF16 / MXFP8) on one GB300 GPU.

Argument marshalling only: every step of the computation runs in the CUDA kernels of the shared
library (include/moebwd.h).  PyTorch provides device memory and streams.  The library is loaded on
first use; if it has not been built, or no CUDA device is present, calls raise -- there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .inputs import (AFFINITY_ON_H, AFFINITY_ON_I, FP8_E4M3, FP8_E5M2, PREC_BF16,  # noqa: F401
                     PREC_MXFP8)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoebwd.so")

QUANT_ROWWISE, QUANT_COLWISE = 0, 1
SF_PLAIN, SF_TILED = 0, 1
STATUS_BAD_EXPERT_ID, STATUS_TIMEOUT, STATUS_BAD_ROUTE_META, STATUS_BAD_SEGMENTS = 1, 2, 4, 8
ACT_CHECKPOINT, ACT_RECOMPUTE, ACT_CHECKPOINT8 = 0, 1, 2
GLU_SWIGLU, GLU_GEGLU = 0, 1
GATE_UP_CONCAT, GATE_UP_INTERLEAVED = 0, 1
DT_BF16, DT_F32 = 0, 1
NORM_LAYER, NORM_RMS = 0, 1

WS_REGIONS = ["EXPERT_OFFSETS", "TILE_OFFSETS", "BLOCK_OFFSETS", "TILE_ROW_FLAT", "FLAT_TILE_ROW",
              "DOUT_G", "DOUT_G_SF", "DOUT_GT", "DOUT_GT_SF", "X_GT", "X_GT_SF", "DH", "DH_SF",
              "DH_T", "DH_T_SF", "AP_T", "AP_T_SF", "DX_EXP", "X_G", "X_G_SF", "GATE_UP_CKPT", "DOUT_Q"]

EXPORTED = ["moe_last_error", "moe_version", "moe_num_blocks_bound", "moe_route_meta_workspace_size",
            "moe_route_meta", "mxfp8_quantize", "moe_bwd_workspace_size", "moe_bwd",
            "moe_bwd_workspace_region", "moe_tile_rows_capacity", "linear_bwd_workspace_size",
            "linear_bwd", "moe_profile_enable", "moe_profile_read", "moe_kernel_launches",
            "moe_route_meta_noalloc", "moe_router_bwd", "moe_set_option", "moe_get_option",
            "moe_balance_workspace_size", "moe_router_fwd", "moe_balance_fwd", "moe_balance_bwd", "moe_glu_fwd",
            "moe_ckpt8_unpack", "layer_norm_fwd", "layer_norm_bwd_workspace_size", "layer_norm_bwd"]

# library options (moe_set_option)
OPTIONS = ["WAIT_LIMIT_NS", "PAIR_GEMMS", "PAIR_TILE_N", "G1_TILE_N", "G2_TILE_N", "G3_TILE_N", "G4_TILE_N",
           "PREP_TILE_ORDER", "G1_GATHER", "G1_WARPS", "PDL", "MN_OPERANDS", "LINEAR_CONCURRENT"]

STAGES = ["route", "prep", "G1_dA_dswiglu", "G3_dW2", "G2_dx_expanded", "G4_dW1", "reduce", "G0_recompute_h"]


class MoeError(RuntimeError):
    pass


class MoeBwdArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("T", "H", "I", "E", "K", "block_size", "precision", "affinity", "fp8_act", "fp8_w",
                 "has_bias")] + \
               [(n, ctypes.c_void_p) for n in
                ("x", "dout", "W1", "W2", "W1_q", "W1_sf", "W2_q", "W2_sf", "b2", "s", "ids",
                 "gate_up_ckpt", "dx", "dW1", "dW2", "ds", "db1", "db2", "status_dev", "workspace")] + \
               [("workspace_bytes", ctypes.c_size_t), ("accumulate", ctypes.c_int), ("act_src", ctypes.c_int)] + \
               [(n, ctypes.c_void_p) for n in ("W1t", "W1t_q", "W1t_sf", "b1", "ds_masked", "num_valid_tokens")] + \
               [(n, ctypes.c_int) for n in ("glu", "gate_up_layout")] + \
               [(n, ctypes.c_void_p) for n in ("intermediate_ckpt", "scaled_intermediate_ckpt", "down_proj_act_ckpt",
                                               "gate_act_ckpt")] + \
               [(n, ctypes.c_void_p) for n in ("expert_offsets", "s_scatter_idx", "block_offsets",
                                               "token_position_to_id", "block_to_expert")] + \
               [(n, ctypes.c_void_p) for n in ("gate_up_ckpt_q", "gate_up_ckpt_sf")]

ROUTE_META_FIELDS = ("expert_offsets", "s_scatter_idx", "block_offsets", "token_position_to_id", "block_to_expert")


_lib = None


def lib():
    """The loaded shared library (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MoeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "moe_last_error": ([], ctypes.c_char_p),
        "moe_version": ([], ctypes.c_char_p),
        "moe_num_blocks_bound": ([i64, i32, i32, i32], i64),
        "moe_route_meta_workspace_size": ([i32, i32, i32, i32], sz),
        "moe_route_meta": ([vp, i32, i32, i32, i32] + [vp] * 10 + [sz, vp], i32),
        "mxfp8_quantize": ([vp, i64, i64, i64, i64, vp, i32, i32, vp, vp, i32, vp], i32),
        "moe_bwd_workspace_size": ([ctypes.POINTER(MoeBwdArgs)], sz),
        "moe_bwd": ([ctypes.POINTER(MoeBwdArgs), vp], i32),
        "moe_bwd_workspace_region": ([ctypes.POINTER(MoeBwdArgs), i32, ctypes.POINTER(sz),
                                      ctypes.POINTER(sz)], i32),
        "moe_tile_rows_capacity": ([i32, i32, i32], i64),
        "linear_bwd_workspace_size": ([i64, i64, i64, i32], sz),
        "linear_bwd": ([vp, vp, vp, i64, i64, i64, i32, i32, vp, vp, vp, sz, vp], i32),
        "moe_profile_enable": ([i32], i32),
        "moe_profile_read": ([ctypes.POINTER(ctypes.c_double), i32, ctypes.POINTER(i32)], i32),
        "moe_kernel_launches": ([], ctypes.c_uint64),
        "moe_route_meta_noalloc": ([vp, i32, i32, i32, i32] + [vp] * 9 + [vp], i32),
        "moe_router_bwd": ([i32, i32, vp, vp, vp, vp, i32, i32, i32, vp, vp], i32),
        "moe_set_option": ([i32, i64], i32),
        "moe_get_option": ([i32], i64),
        "moe_balance_workspace_size": ([i32] * 4, sz),
        "moe_router_fwd": ([i32, i32, vp, i64, i32, i32, i32, vp, i32, f32, f32] + [vp] * 8 + [sz, vp], i32),
        "moe_balance_fwd": ([vp, i64, vp, i32, i32, i32, vp, i32, f32, f32] + [vp] * 6 + [sz, vp], i32),
        "moe_balance_bwd": ([vp, i64, vp, vp, i32, i32, i32, vp, i32, f32, f32, vp, vp, i64, vp, vp, vp], i32),
        "moe_glu_fwd": ([vp, i64, i64, i32, i32, i32, i64, i32, i32] + [vp] * 5 + [i64, vp, vp, vp, vp], i32),
        "moe_ckpt8_unpack": ([vp, vp, i64, i32, i32, i32, i64, i32, vp, vp, vp, vp, i64, vp], i32),
        "layer_norm_fwd": ([i32, vp, i64, vp, i64, vp, vp, i32, i32, i64, i64, f32, vp, vp, vp, vp, vp], i32),
        "layer_norm_bwd_workspace_size": ([i64, i64], sz),
        "layer_norm_bwd": ([i32, vp, i64, vp, i64, vp, vp, vp, vp, i64, i32, i32, i64, i64, vp, vp, vp, i32, vp, sz,
                            vp], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != 0:
        raise MoeError(f"{what} failed ({rc}): {lib().moe_last_error().decode()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:  # the current stream of the current device
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise MoeError("tensors must be CUDA tensors (there is no CPU path)")
        if t is not None and not t.is_contiguous():
            raise MoeError("tensors must be contiguous")


def profile_enable(enable: bool = True):
    """Start (or stop) recording per-stage CUDA events inside moe_bwd; discards earlier records."""
    _check(lib().moe_profile_enable(int(enable)), "moe_profile_enable")


def profile_read() -> tuple[dict, int]:
    """Total milliseconds per stage over the profiled moe_bwd calls, and the number of calls."""
    arr = (ctypes.c_double * len(STAGES))()
    calls = ctypes.c_int()
    _check(lib().moe_profile_read(arr, len(STAGES), ctypes.byref(calls)), "moe_profile_read")
    return {n: arr[i] for i, n in enumerate(STAGES)}, calls.value


def set_option(name: str, value: int | None):
    """Set a library option by its name in OPTIONS (None restores the default)."""
    _check(lib().moe_set_option(OPTIONS.index(name), -1 if value is None else int(value)), "moe_set_option")


def get_option(name: str) -> int:
    return int(lib().moe_get_option(OPTIONS.index(name)))


class option:
    """Context manager: set a library option for the duration of a block, then restore its old value."""

    def __init__(self, name: str, value: int):
        self.name, self.value = name, value

    def __enter__(self):
        self.old = get_option(self.name)
        set_option(self.name, self.value)
        return self

    def __exit__(self, *exc):
        set_option(self.name, self.old)
        return False


def kernel_launches() -> int:
    """Kernels launched by the library so far in this process."""
    return int(lib().moe_kernel_launches())


def num_blocks_bound(T: int, K: int, E: int, block_size: int) -> int:
    return int(lib().moe_num_blocks_bound(T, K, E, block_size))


def tile_rows_capacity(T: int, K: int, E: int) -> int:
    return int(lib().moe_tile_rows_capacity(T, K, E))


def _ws(nbytes: int, device):
    # 256-byte aligned by the CUDA caching allocator
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def route_meta(ids: torch.Tensor, E: int, block_size: int, stream=None) -> dict:
    """moe_route_meta on int32 ids [T,K]; returns the metadata tensors and the status word."""
    _need_cuda(ids)
    assert ids.dtype == torch.int32 and ids.dim() == 2
    T, K = ids.shape
    dev = ids.device
    N = num_blocks_bound(T, K, E, block_size)
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(expert_offsets=torch.empty(E + 1, **i32), x_gather_idx=torch.full((T * K,), -1, **i32),
               s_scatter_idx=torch.full((T * K,), -1, **i32), s_reverse_scatter_idx=torch.empty(T * K, **i32),
               token_position_to_id=torch.empty(max(N * block_size, 1), **i32),
               block_to_expert=torch.empty(max(N, 1), **i32), block_offsets=torch.empty(E + 1, **i32),
               num_blocks=torch.empty(1, **i32), status=torch.empty(1, **i32))
    wsz = lib().moe_route_meta_workspace_size(T, K, E, block_size)
    ws = _ws(wsz, dev)
    rc = lib().moe_route_meta(_ptr(ids), T, K, E, block_size, *[_ptr(out[k]) for k in (
        "expert_offsets", "x_gather_idx", "s_scatter_idx", "s_reverse_scatter_idx", "token_position_to_id",
        "block_to_expert", "block_offsets", "num_blocks", "status")], _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "moe_route_meta")
    out["token_position_to_id"] = out["token_position_to_id"][: N * block_size]
    out["block_to_expert"] = out["block_to_expert"][:N]
    out["_workspace"] = ws
    return out


def sf_bytes(rows: int, cols: int, scale_layout: int) -> int:
    """Scale bytes of an [rows, cols] matrix quantised along cols."""
    if scale_layout == SF_TILED:
        return ((rows + 127) // 128) * ((cols + 127) // 128) * 512
    return rows * (cols // 32)


def mxfp8_quantize(x: torch.Tensor, axis: int = QUANT_ROWWISE, fmt: int = FP8_E5M2,
                   row_index: torch.Tensor | None = None, scale_layout: int = SF_TILED, stream=None):
    """mxfp8_quantize on a bf16 [src_rows, cols] tensor.  Returns (codes uint8, scales uint8).
    ROWWISE: codes [rows, cols]; COLWISE: codes of the transposed matrix [cols, rows]."""
    _need_cuda(x, row_index)
    assert x.dtype == torch.bfloat16 and x.dim() == 2
    src_rows, cols = x.shape
    rows = row_index.numel() if row_index is not None else src_rows
    if axis == QUANT_ROWWISE:
        q = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
        sf = torch.zeros(sf_bytes(rows, cols, scale_layout), dtype=torch.uint8, device=x.device)
    else:
        q = torch.empty(cols, rows, dtype=torch.uint8, device=x.device)
        sf = torch.zeros(sf_bytes(cols, rows, scale_layout), dtype=torch.uint8, device=x.device)
    rc = lib().mxfp8_quantize(_ptr(x), src_rows, rows, cols, cols, _ptr(row_index), axis, fmt, _ptr(q),
                              _ptr(sf), scale_layout, _stream(stream))
    _check(rc, "mxfp8_quantize")
    return q, sf


def quantize_weights(W: torch.Tensor, fmt: int = FP8_E4M3, stream=None):
    """Pre-quantise expert weights [E, R, C] along C (the contraction of their GEMM) as the [E*R, C]
    matrix with tiled scales, the layout moe_bwd expects for W1_q/W1_sf, W2_q/W2_sf and (given the
    per-expert transpose of W1) W1t_q/W1t_sf."""
    E, R, C = W.shape
    return mxfp8_quantize(W.reshape(E * R, C), QUANT_ROWWISE, fmt, None, SF_TILED, stream)


def _check_status(t, device):
    """Refuses a status word that the kernels on `device` cannot write: anything but one int32 there."""
    if not t.is_cuda or t.dtype is not torch.int32 or t.numel() != 1:
        raise MoeError(f"status must be a CUDA tensor of one int32, got {t.dtype} {tuple(t.shape)} on {t.device}")
    here = device.index if device.index is not None else torch.cuda.current_device()
    if device.type != "cuda" or t.device.index != here:
        raise MoeError(f"status is on {t.device}, which is not the operator's device")


class MoeBwd:
    """One MoE backward problem bound to device buffers: outputs and workspace are allocated once,
    run() enqueues moe_bwd on the stream (no host synchronisation)."""

    def __init__(self, *, T, H, I, E, K, block_size, precision=PREC_BF16, affinity=AFFINITY_ON_H,
                 fp8_act=FP8_E5M2, fp8_w=FP8_E4M3, has_bias=False, accumulate=False, act_src=ACT_CHECKPOINT,
                 ds_masked=False, glu=GLU_SWIGLU, gate_up_layout=GATE_UP_CONCAT, device="cuda", status=None):
        """status: an int32 [1] CUDA tensor on `device` for the status word (None: one is made, 0 until the first run)."""
        self.device = torch.device(device)
        if status is not None:
            _check_status(status, self.device)
        self.a = MoeBwdArgs()
        self.a.glu = int(glu)
        self.a.gate_up_layout = int(gate_up_layout)
        self.a.accumulate = int(bool(accumulate))
        self.a.act_src = int(act_src)
        for k, v in dict(T=T, H=H, I=I, E=E, K=K, block_size=block_size, precision=precision,
                         affinity=affinity, fp8_act=fp8_act, fp8_w=fp8_w, has_bias=int(bool(has_bias))).items():
            setattr(self.a, k, int(v))
        size = lib().moe_bwd_workspace_size(ctypes.byref(self.a))
        if size == 0:
            raise MoeError(f"unsupported moe_bwd configuration: {lib().moe_last_error().decode()}")
        self.workspace = _ws(size, self.device)
        dev = self.device
        self.dx = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        self.dW1 = torch.empty(E, H, 2 * I, dtype=torch.bfloat16, device=dev)
        self.dW2 = torch.empty(E, I, H, dtype=torch.bfloat16, device=dev)
        self.ds = torch.empty(T, K, dtype=torch.float32, device=dev)
        self.db1 = torch.empty(E, 2 * I, dtype=torch.float32, device=dev) if has_bias else None
        self.db2 = torch.empty(E, H, dtype=torch.float32, device=dev) if has_bias else None
        self.ds_masked = torch.empty(T * E, dtype=torch.float32, device=dev) if ds_masked else None
        self.status = torch.zeros(1, dtype=torch.int32, device=dev) if status is None else status
        self._keep = []

    def bind(self, *, x, dout, s, ids, ckpt=None, ckpt_q=None, ckpt_sf=None, W1=None, W2=None, W1_q=None, W1_sf=None, W2_q=None, W2_sf=None,
             b2=None, W1t=None, W1t_q=None, W1t_sf=None, b1=None, num_valid_tokens=None, intermediate_ckpt=None,
             scaled_intermediate_ckpt=None, down_proj_act_ckpt=None, gate_act_ckpt=None, route_meta=None):
        """ckpt: the [N,2,I,B] checkpoint (act_src ACT_CHECKPOINT); ckpt_q, ckpt_sf: its 8-bit form, as
        glu_fwd returns it (act_src ACT_CHECKPOINT8).  W1t (bf16 [E,2I,H]) or W1t_q/W1t_sf
        and optionally b1 [E,2I]: the operands of the recomputation (act_src ACT_RECOMPUTE).
        intermediate_ckpt / scaled_intermediate_ckpt / gate_act_ckpt [N,I,B] and down_proj_act_ckpt
        [N,B,H] (bf16, block layout): saved forward values, see the MoeBwdArgs fields.
        route_meta: routing metadata from the caller (a dict with int32 CUDA tensors expert_offsets,
        s_scatter_idx, block_offsets and optionally token_position_to_id, block_to_expert -- e.g.
        route_meta()'s result); None: moe_bwd computes it from ids."""
        _need_cuda(x, dout, s, ids, ckpt, W1, W2, W1_q, W1_sf, W2_q, W2_sf, b2, W1t, W1t_q, W1t_sf, b1, num_valid_tokens,
                   intermediate_ckpt, scaled_intermediate_ckpt, down_proj_act_ckpt, gate_act_ckpt, ckpt_q, ckpt_sf)
        if num_valid_tokens is not None:
            assert num_valid_tokens.dtype == torch.int32 and num_valid_tokens.numel() == 1
        a = self.a
        Nb = num_blocks_bound(a.T, a.K, a.E, a.block_size)
        for t in (intermediate_ckpt, scaled_intermediate_ckpt, gate_act_ckpt):
            assert t is None or (t.dtype == torch.bfloat16 and tuple(t.shape) == (Nb, a.I, a.block_size))
        assert down_proj_act_ckpt is None or (down_proj_act_ckpt.dtype == torch.bfloat16 and
                                              tuple(down_proj_act_ckpt.shape) == (Nb, a.block_size, a.H))
        assert x.dtype == torch.bfloat16 and dout.dtype == torch.bfloat16
        assert s.dtype == torch.float32 and ids.dtype == torch.int32
        assert tuple(x.shape) == (a.T, a.H) and tuple(dout.shape) == (a.T, a.H)
        assert tuple(s.shape) == (a.T, a.K) and tuple(ids.shape) == (a.T, a.K)
        if ckpt is not None:
            assert ckpt.dtype == torch.bfloat16
            assert tuple(ckpt.shape) == (Nb, 2, a.I, a.block_size), (tuple(ckpt.shape), Nb)
        if ckpt_q is not None:
            assert ckpt_q.dtype == torch.int8 and tuple(ckpt_q.shape) == (Nb, 2, a.I, a.block_size)
        if ckpt_sf is not None:
            assert ckpt_sf.dtype == torch.uint8 and tuple(ckpt_sf.shape) == ckpt8_sf_shape(Nb, a.I, a.block_size)
        if W1t is not None:
            assert W1t.dtype == torch.bfloat16 and tuple(W1t.shape) == (a.E, 2 * a.I, a.H)
        if b1 is not None:
            assert b1.dtype == torch.bfloat16 and tuple(b1.shape) == (a.E, 2 * a.I)
        for name, t in dict(x=x, dout=dout, s=s, ids=ids, gate_up_ckpt=ckpt, W1=W1, W2=W2, W1_q=W1_q,
                            W1_sf=W1_sf, W2_q=W2_q, W2_sf=W2_sf, b2=b2, W1t=W1t, W1t_q=W1t_q, W1t_sf=W1t_sf,
                            b1=b1, num_valid_tokens=num_valid_tokens, intermediate_ckpt=intermediate_ckpt,
                            scaled_intermediate_ckpt=scaled_intermediate_ckpt,
                            down_proj_act_ckpt=down_proj_act_ckpt, gate_act_ckpt=gate_act_ckpt,
                            gate_up_ckpt_q=ckpt_q, gate_up_ckpt_sf=ckpt_sf).items():
            setattr(a, name, None if t is None else t.data_ptr())
        for name in ("dx", "dW1", "dW2", "ds", "db1", "db2", "ds_masked", "status"):
            t = getattr(self, name)
            setattr(a, "status_dev" if name == "status" else name, None if t is None else t.data_ptr())
        rm = {k: route_meta.get(k) if route_meta else None for k in ROUTE_META_FIELDS}
        for k, t in rm.items():
            if t is not None:
                _need_cuda(t)
                assert t.dtype == torch.int32, k
            setattr(a, k, None if t is None else t.data_ptr())
        a.workspace = self.workspace.data_ptr()
        a.workspace_bytes = self.workspace.numel()
        self._keep = [x, dout, s, ids, ckpt, W1, W2, W1_q, W1_sf, W2_q, W2_sf, b2, W1t, W1t_q, W1t_sf, b1,
                      num_valid_tokens, intermediate_ckpt, scaled_intermediate_ckpt, down_proj_act_ckpt, gate_act_ckpt,
                      ckpt_q, ckpt_sf, *rm.values()]
        return self

    def run(self, stream=None):
        _check(lib().moe_bwd(ctypes.byref(self.a), _stream(stream)), "moe_bwd")
        return self

    def outputs(self) -> dict:
        return dict(dx=self.dx, dW1=self.dW1, dW2=self.dW2, ds=self.ds, db1=self.db1, db2=self.db2,
                    ds_masked=self.ds_masked, status=self.status)

    def region(self, name: str) -> torch.Tensor:
        """Bytes of one workspace region (see MOE_WS_* in include/moebwd.h)."""
        off, nb = ctypes.c_size_t(), ctypes.c_size_t()
        rc = lib().moe_bwd_workspace_region(ctypes.byref(self.a), WS_REGIONS.index(name), ctypes.byref(off),
                                            ctypes.byref(nb))
        _check(rc, "moe_bwd_workspace_region")
        return self.workspace[off.value: off.value + nb.value]

    @property
    def tile_rows(self) -> int:
        return tile_rows_capacity(self.a.T, self.a.K, self.a.E)


def moe_bwd(*, x, dout, s, ids, E, I, block_size, ckpt=None, ckpt_q=None, ckpt_sf=None, W1=None, W2=None, W1_q=None, W1_sf=None, W2_q=None,
            W2_sf=None, b2=None, W1t=None, W1t_q=None, W1t_sf=None, b1=None, precision=PREC_BF16,
            affinity=AFFINITY_ON_H, fp8_act=FP8_E5M2, fp8_w=FP8_E4M3, accumulate=False, stream=None) -> dict:
    """One-shot MoE backward (allocates outputs and workspace).  Returns dx, dW1, dW2, ds, db1, db2
    and the device status word (nonzero: invalid expert ids or a pipeline timeout).  The gate/up
    pre-activations come from ckpt, from its 8-bit form ckpt_q/ckpt_sf, or, with neither, from a
    recomputation of x and W1t (or W1t_q/W1t_sf) plus b1."""
    T, H = x.shape
    K = ids.shape[1]
    op = MoeBwd(T=T, H=H, I=I, E=E, K=K, block_size=block_size, precision=precision, affinity=affinity,
                fp8_act=fp8_act, fp8_w=fp8_w, has_bias=b2 is not None, accumulate=accumulate,
                act_src=(ACT_CHECKPOINT if ckpt is not None else ACT_CHECKPOINT8 if ckpt_q is not None
                         else ACT_RECOMPUTE), device=x.device,
                status=torch.empty(1, dtype=torch.int32, device=x.device))  # the call itself resets it
    op.bind(x=x, dout=dout, s=s, ids=ids, ckpt=ckpt, ckpt_q=ckpt_q, ckpt_sf=ckpt_sf, W1=W1, W2=W2, W1_q=W1_q, W1_sf=W1_sf, W2_q=W2_q,
            W2_sf=W2_sf, b2=b2, W1t=W1t, W1t_q=W1t_q, W1t_sf=W1t_sf, b1=b1).run(stream)
    out = op.outputs()
    out["_op"] = op
    return out


ROUTER_SOFTMAX_OVER_TOPK, ROUTER_TOPK_OVER_SOFTMAX, ROUTER_TOPK = 0, 1, 2


def router_bwd(mode: int, ids: torch.Tensor, dscores: torch.Tensor, E: int, logits=None, scores=None,
               renorm: bool = False, stream=None) -> torch.Tensor:
    """moe_router_bwd: gradient of the router logits [T, E] from the scores' gradient [T, K]."""
    _need_cuda(ids, dscores, logits, scores)
    T, K = ids.shape
    out = torch.empty(T, E, dtype=torch.float32, device=ids.device)
    rc = lib().moe_router_bwd(mode, int(renorm), _ptr(logits), _ptr(scores), _ptr(dscores), _ptr(ids), T, K, E,
                              _ptr(out), _stream(stream))
    _check(rc, "moe_router_bwd")
    return out


def _refuse(t, dtype, shape, name, dev, how):
    if not t.is_cuda or t.device != dev:
        raise MoeError(f"{name} must be a CUDA tensor on {dev} (there is no CPU path)")
    raise MoeError(f"{name} must be {dtype} {shape} {how}, got {t.dtype} {tuple(t.shape)} of strides {t.stride()}")


def _rows(t, dtype, shape, name, dev):
    """Row stride of a 2-D CUDA tensor of this type and shape whose rows are dense; raises on anything else."""
    if t.device != dev or not t.is_cuda or t.dtype is not dtype or t.shape != shape:
        _refuse(t, dtype, shape, name, dev, "with dense rows")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        _refuse(t, dtype, shape, name, dev, "with dense rows")
    return ld if shape[0] > 1 else max(ld, shape[1])


def _dense(t, dtype, shape, name, dev):
    """Pointer of a dense CUDA tensor of this type and shape, None for None; raises on anything else."""
    if t is None:
        return None
    if t.device != dev or not t.is_cuda or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _refuse(t, dtype, shape, name, dev, "and contiguous")
    return t.data_ptr()


def _here(dev):
    """Handle of the current stream of the tensors' device, which has to be the current one.  What a call allocates
    belongs to that stream, so that nothing else is given its memory while the call may still use it; with a
    `stream` argument a call therefore runs with that stream made current.  Tensors made on another stream are
    the caller's to order (Stream.wait_stream) and to keep."""
    if dev.type != "cuda":
        raise MoeError("tensors must be CUDA tensors (there is no CPU path)")
    if dev.index != torch._C._cuda_getDevice():
        raise MoeError(f"tensors are on {dev}, which is not the current device")
    return torch._C._cuda_getCurrentRawStream(dev.index)


try:  # the allocator's entry point without torch.empty's argument parsing (0.9 us instead of 1.6 us a tensor)
    from torch._C._dynamo.guards import _empty_strided_cuda as _empty_strided
except ImportError:
    def _empty_strided(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _new1(n, dtype):
    """A vector on the current device (_here checked that it is the tensors')."""
    return _empty_strided((n,), (1,), dtype)


def _new2(rows, cols, dtype):
    """A dense matrix on the current device."""
    return _empty_strided((rows, cols), (cols, 1), dtype)


_DT = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}


def _norm_types(x, gamma, what):
    if x.dim() != 2:
        raise MoeError(f"{what}: x must be [T, H]")
    if x.dtype not in _DT or gamma.dtype not in _DT:
        raise MoeError(f"{what}: rows and weights must be bfloat16 or float32")
    return x.shape[0], x.shape[1], x.device


def layer_norm_fwd(x, gamma, beta=None, eps: float = 1e-5, residual=None, kind: int = NORM_LAYER, stream=None) -> dict:
    """layer_norm_fwd on rows x [T, H] (bf16 or fp32, dense rows of any stride), plus `residual` when given.
    Returns y, mean (NORM_LAYER, else None), rstd, and sum = x + residual (None without a residual), the
    rows that layer_norm_bwd takes as its x.  gamma, beta [H] in bf16 or fp32."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return layer_norm_fwd(x, gamma, beta, eps, residual, kind)
    T, H, dev = _norm_types(x, gamma, "layer_norm_fwd")
    ldx = _rows(x, x.dtype, (T, H), "x", dev)
    ldr = 0 if residual is None else _rows(residual, x.dtype, (T, H), "residual", dev)
    g, b = _dense(gamma, gamma.dtype, (H,), "gamma", dev), _dense(beta, gamma.dtype, (H,), "beta", dev)
    st = _here(dev)
    y = _new2(T, H, x.dtype)
    total = None if residual is None else _new2(T, H, x.dtype)
    rstd = _new1(T, torch.float32)
    mean = _new1(T, torch.float32) if kind == NORM_LAYER else None
    rc = lib().layer_norm_fwd(kind, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, g, b,
                              _DT[x.dtype], _DT[gamma.dtype], T, H, eps, y.data_ptr(),
                              None if total is None else total.data_ptr(),
                              None if mean is None else mean.data_ptr(), rstd.data_ptr(), st)
    _check(rc, "layer_norm_fwd")
    return dict(y=y, mean=mean, rstd=rstd, sum=total)


def layer_norm_bwd(dy, x, gamma, mean, rstd, dres=None, kind: int = NORM_LAYER, dbeta: bool = True,
                   accumulate_into=None, stream=None) -> dict:
    """layer_norm_bwd: dx (plus `dres`, the gradient that reaches the rows past the norm), dgamma and, with a
    mean and unless dbeta is False, dbeta, in fp32.  x are the normalised rows (with a residual: the forward's
    sum).  accumulate_into: an earlier result whose dgamma and dbeta are added to in place."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return layer_norm_bwd(dy, x, gamma, mean, rstd, dres, kind, dbeta, accumulate_into)
    T, H, dev = _norm_types(x, gamma, "layer_norm_bwd")
    ldx, lddy = _rows(x, x.dtype, (T, H), "x", dev), _rows(dy, x.dtype, (T, H), "dy", dev)
    ldres = 0 if dres is None else _rows(dres, x.dtype, (T, H), "dres", dev)
    g, r = _dense(gamma, gamma.dtype, (H,), "gamma", dev), _dense(rstd, torch.float32, (T,), "rstd", dev)
    m = _dense(mean, torch.float32, (T,), "mean", dev) if kind == NORM_LAYER else None
    st = _here(dev)
    dx = _new2(T, H, x.dtype)
    if accumulate_into is not None:
        dg, db = accumulate_into["dgamma"], accumulate_into["dbeta"]
        _dense(dg, torch.float32, (H,), "dgamma", dev)
        _dense(db, torch.float32, (H,), "dbeta", dev)
    else:
        dg = _new1(H, torch.float32)
        db = _new1(H, torch.float32) if dbeta and kind == NORM_LAYER else None
    ws = _new1(max(lib().layer_norm_bwd_workspace_size(T, H), 256), torch.uint8)
    rc = lib().layer_norm_bwd(kind, dy.data_ptr(), lddy, x.data_ptr(), ldx, g, m, r,
                              None if dres is None else dres.data_ptr(), ldres, _DT[x.dtype], _DT[gamma.dtype], T, H,
                              dx.data_ptr(), dg.data_ptr(), None if db is None else db.data_ptr(),
                              int(accumulate_into is not None), ws.data_ptr(), ws.numel(), st)
    _check(rc, "layer_norm_bwd")
    return dict(dx=dx, dgamma=dg, dbeta=db)


def _segments(seg_offsets, dev):
    if seg_offsets is None:
        return None, 1
    if seg_offsets.dim() != 1 or seg_offsets.numel() < 2:
        raise MoeError("seg_offsets must be int32 [num_seq + 1]")
    n = seg_offsets.numel()
    return _dense(seg_offsets, torch.int32, (n,), "seg_offsets", dev), n - 1


def _balance_outputs(T, K, E, S, dev):
    return (_new2(S, E, torch.int32), _new2(S, E, torch.float32),
            _new1(2, torch.float32), _new1(1, torch.int32),
            _new1(max(lib().moe_balance_workspace_size(T, K, E, S), 256), torch.uint8))


def router_fwd(mode: int, logits: torch.Tensor, K: int, renorm: bool = False, seg_offsets=None, alpha: float = 0.0,
               beta: float = 0.0, balance: bool = True, stream=None) -> dict:
    """moe_router_fwd: top-K of fp32 logits [T, E] (dense rows of any stride).  Returns scores [T, K], ids [T, K],
    lse [T] and, unless balance is False, counts and prob_sum [num_seq, E], loss [2] = (balance, z).  With the losses or
    with seg_offsets also status, int32 [1]: STATUS_BAD_SEGMENTS for bad offsets (the results are then invalid)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return router_fwd(mode, logits, K, renorm, seg_offsets, alpha, beta, balance)
    if logits.dim() != 2:
        raise MoeError("logits must be [T, E]")
    T, E = logits.shape
    dev = logits.device
    ld = _rows(logits, torch.float32, (T, E), "logits", dev)
    off, S = _segments(seg_offsets, dev)
    st = _here(dev)
    scores = _new2(T, K, torch.float32)
    ids = _new2(T, K, torch.int32)
    out = dict(scores=scores, ids=ids, lse=_new1(T, torch.float32))
    p = [None] * 4
    ws = None
    if balance:
        counts, prob, loss, status, ws = _balance_outputs(T, K, E, S, dev)
        out.update(counts=counts, prob_sum=prob, loss=loss, status=status)
        p = [counts.data_ptr(), prob.data_ptr(), loss.data_ptr(), status.data_ptr()]
    elif off is not None:
        out["status"] = _new1(1, torch.int32)
        p[3] = out["status"].data_ptr()
    rc = lib().moe_router_fwd(mode, int(renorm), logits.data_ptr(), ld, T, K, E, off, S, alpha, beta,
                              scores.data_ptr(), ids.data_ptr(), out["lse"].data_ptr(), *p,
                              None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), st)
    _check(rc, "moe_router_fwd")
    return out


def balance_fwd(logits: torch.Tensor, ids: torch.Tensor, seg_offsets=None, alpha: float = 0.0, beta: float = 0.0,
                stream=None) -> dict:
    """moe_balance_fwd: the losses of router_fwd for ids [T, K] selected elsewhere.  Returns lse, counts, prob_sum,
    loss and status."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return balance_fwd(logits, ids, seg_offsets, alpha, beta)
    if logits.dim() != 2 or ids.dim() != 2:
        raise MoeError("logits must be [T, E] and ids [T, K]")
    (T, E), K, dev = logits.shape, ids.shape[1], logits.device
    ld = _rows(logits, torch.float32, (T, E), "logits", dev)
    idp = _dense(ids, torch.int32, (T, K), "ids", dev)
    off, S = _segments(seg_offsets, dev)
    st = _here(dev)
    lse = _new1(T, torch.float32)
    counts, prob, loss, status, ws = _balance_outputs(T, K, E, S, dev)
    rc = lib().moe_balance_fwd(logits.data_ptr(), ld, idp, T, K, E, off, S, alpha, beta, lse.data_ptr(),
                               counts.data_ptr(), prob.data_ptr(), loss.data_ptr(), status.data_ptr(),
                               ws.data_ptr(), ws.numel(), st)
    _check(rc, "moe_balance_fwd")
    return dict(lse=lse, counts=counts, prob_sum=prob, loss=loss, status=status)


def balance_bwd(logits: torch.Tensor, lse: torch.Tensor, counts: torch.Tensor, K: int, seg_offsets=None,
                alpha: float = 0.0, beta: float = 0.0, dloss=None, add=None, stream=None, status=None) -> torch.Tensor:
    """moe_balance_bwd: gradient of dloss[0] * balance + dloss[1] * z by the logits [T, E], plus `add` (e.g.
    router_bwd's result).  lse and counts are the forward's.  status: an int32 [1] CUDA tensor that the call sets to 0, or
    to STATUS_BAD_SEGMENTS for bad offsets (the result is then invalid; the forward's status reports the same offsets)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return balance_bwd(logits, lse, counts, K, seg_offsets, alpha, beta, dloss, add, None, status)
    if logits.dim() != 2:
        raise MoeError("logits must be [T, E]")
    T, E = logits.shape
    dev = logits.device
    ld = _rows(logits, torch.float32, (T, E), "logits", dev)
    ld_add = 0 if add is None else _rows(add, torch.float32, (T, E), "add", dev)
    off, S = _segments(seg_offsets, dev)
    lp, cp = _dense(lse, torch.float32, (T,), "lse", dev), _dense(counts, torch.int32, (S, E), "counts", dev)
    dl = _dense(dloss, torch.float32, (2,), "dloss", dev)
    sp = _dense(status, torch.int32, (1,), "status", dev)
    st = _here(dev)
    out = _new2(T, E, torch.float32)
    rc = lib().moe_balance_bwd(logits.data_ptr(), ld, lp, cp, T, K, E, off, S, alpha, beta, dl,
                               None if add is None else add.data_ptr(), ld_add, out.data_ptr(), sp, st)
    _check(rc, "moe_balance_bwd")
    return out


def ckpt8_sf_shape(N: int, I: int, block_size: int) -> tuple:
    """Shape of the scale bytes of an 8-bit checkpoint: 128-slot tile, 32 features, 32-slot group, feature."""
    return (N, 2, block_size // 128, I // 32, 4, 32)


def _meta_ptrs(route_meta, dev):
    eo, bo, b2e = route_meta["expert_offsets"], route_meta["block_offsets"], route_meta["block_to_expert"]
    E, N = eo.numel() - 1, b2e.numel()
    return (_dense(eo, torch.int32, (E + 1,), "expert_offsets", dev), _dense(bo, torch.int32, (E + 1,), "block_offsets", dev),
            _dense(b2e, torch.int32, (N,), "block_to_expert", dev), E, N)


def glu_fwd(h: torch.Tensor, route_meta: dict, block_size: int, glu: int = GLU_SWIGLU,
            gate_up_layout: int = GATE_UP_CONCAT, s=None, checkpoint: bool = True, stream=None) -> dict:
    """moe_glu_fwd on the grouped rows h bf16 [rows, 2I]: a = act(gate) * up [rows, I] (times the row's score
    with s [T, K], whose s_scatter_idx route_meta then holds) and, unless checkpoint is False, the 8-bit
    checkpoint ckpt_q [N, 2, I, B], ckpt_sf for moe_bwd.  route_meta: route_meta()'s dict."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return glu_fwd(h, route_meta, block_size, glu, gate_up_layout, s, checkpoint)
    if h.dim() != 2 or h.shape[1] % 2:
        raise MoeError("h must be [rows, 2I]")
    rows, I, dev = h.shape[0], h.shape[1] // 2, h.device
    ldh = _rows(h, torch.bfloat16, (rows, 2 * I), "h", dev)
    eo, bo, b2e, E, N = _meta_ptrs(route_meta, dev)
    sp = sip = None
    slots = 0
    if s is not None:
        slots = s.numel()
        sp = _dense(s, torch.float32, tuple(s.shape), "s", dev)
        idx = route_meta["s_scatter_idx"]
        if idx.numel() < rows:
            raise MoeError("s_scatter_idx is shorter than the rows of h")
        sip = _dense(idx, torch.int32, tuple(idx.shape), "s_scatter_idx", dev)
    st = _here(dev)
    a = _new2(rows, I, torch.bfloat16)
    q = sf = None
    if checkpoint:
        q = _empty_strided((N, 2, I, block_size), (2 * I * block_size, I * block_size, block_size, 1), torch.int8)
        per = 4 * I                                     # scale bytes of 128 slots
        sf = _empty_strided(ckpt8_sf_shape(N, I, block_size),
                            (2 * (block_size // 128) * per, (block_size // 128) * per, per, 128, 32, 1), torch.uint8)
    rc = lib().moe_glu_fwd(h.data_ptr(), ldh, rows, I, E, block_size, N, glu, gate_up_layout, eo, bo, b2e, sp, sip,
                           slots, a.data_ptr(), None if q is None else q.data_ptr(),
                           None if sf is None else sf.data_ptr(), st)
    _check(rc, "moe_glu_fwd")
    return dict(a=a, ckpt_q=q, ckpt_sf=sf)


def ckpt8_unpack(ckpt_q: torch.Tensor, ckpt_sf: torch.Tensor, route_meta: dict, rows: int,
                 gate_up_layout: int = GATE_UP_CONCAT, stream=None) -> torch.Tensor:
    """moe_ckpt8_unpack: the 8-bit checkpoint's values as grouped rows bf16 [rows, 2I] (rows that no expert has
    are left unwritten)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ckpt8_unpack(ckpt_q, ckpt_sf, route_meta, rows, gate_up_layout)
    if ckpt_q.dim() != 4:
        raise MoeError("ckpt_q must be [N, 2, I, B]")
    N, _, I, B = ckpt_q.shape
    dev = ckpt_q.device
    eo, bo, b2e, E, Nb = _meta_ptrs(route_meta, dev)
    qp = _dense(ckpt_q, torch.int8, (Nb, 2, I, B), "ckpt_q", dev)
    sp = _dense(ckpt_sf, torch.uint8, ckpt8_sf_shape(N, I, B), "ckpt_sf", dev)
    st = _here(dev)
    h = _new2(rows, 2 * I, torch.bfloat16)
    rc = lib().moe_ckpt8_unpack(qp, sp, rows, I, E, B, Nb, gate_up_layout, eo, bo, b2e, h.data_ptr(), 2 * I, st)
    _check(rc, "moe_ckpt8_unpack")
    return h


class LinearBwd:
    """Dense linear backward dX = dY @ W, dW = dY^T @ X with buffers allocated once."""

    def __init__(self, M, N, K, precision=PREC_MXFP8, fp8=FP8_E5M2, device="cuda"):
        self.M, self.N, self.K, self.precision, self.fp8 = M, N, K, precision, fp8
        dev = torch.device(device)
        self.workspace = _ws(lib().linear_bwd_workspace_size(M, N, K, precision), dev)
        self.dX = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
        self.dW = torch.empty(N, K, dtype=torch.bfloat16, device=dev)

    def run(self, dY, W, X, stream=None):
        _need_cuda(dY, W, X)
        rc = lib().linear_bwd(_ptr(dY), _ptr(W), _ptr(X), self.M, self.N, self.K, self.precision, self.fp8,
                              _ptr(self.dX), _ptr(self.dW), _ptr(self.workspace), self.workspace.numel(),
                              _stream(stream))
        _check(rc, "linear_bwd")
        return self


def linear_bwd(dY, W, X, precision=PREC_MXFP8, fp8=FP8_E5M2, stream=None):
    M, N = dY.shape
    K = X.shape[1]
    op = LinearBwd(M, N, K, precision, fp8, dY.device).run(dY, W, X, stream)
    return dict(dX=op.dX, dW=op.dW)
