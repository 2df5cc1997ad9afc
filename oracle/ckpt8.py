"""Oracle: the 8-bit gate/up checkpoint and the forward's gated activation (test infrastructure only).

Codes and scale bytes from the definition, one group of 32 consecutive slots of one feature at a time:
byte = max(1, exponent field of the largest magnitude - 6), code = the integer nearest to v / 2^(byte - 127)
(ties to even) within +-127, value = code 2^(byte - 127); a group with a NaN or an infinity: byte 255, values
NaN.  Scale bytes are laid out [N, 2, B/128, I/32, 4, 32].
"""
from __future__ import annotations

import math

import numpy as np

from oracle.moe import gelu


def group_codes(v):
    """(codes, byte) of one group of fp32-representable values."""
    v = np.asarray(v, dtype=np.float64)
    if not np.all(np.isfinite(v)):
        return np.zeros(len(v), dtype=np.int64), 255
    m = np.max(np.abs(v))
    field = 0 if m < 2.0 ** -126 else math.frexp(m)[1] - 1 + 127
    byte = max(1, field - 6)
    return np.clip(np.rint(v * 2.0 ** (127 - byte)), -127, 127).astype(np.int64), byte


def pack(ckpt):
    """int8 codes [N, 2, I, B] and scale bytes [N, 2, B/128, I/32, 4, 32] of a checkpoint [N, 2, I, B]."""
    N, two, I, B = ckpt.shape
    q = np.zeros((N, two, I, B), dtype=np.int8)
    sf = np.zeros((N, two, B // 128, I // 32, 4, 32), dtype=np.uint8)
    for n in range(N):
        for w in range(two):
            for i in range(I):
                for g in range(B // 32):
                    c, byte = group_codes(ckpt[n, w, i, 32 * g:32 * g + 32])
                    q[n, w, i, 32 * g:32 * g + 32] = c
                    sf[n, w, g // 4, i // 32, g % 4, i % 32] = byte
    return q, sf


def unpack(q, sf):
    """The values [N, 2, I, B]."""
    N, two, I, B = q.shape
    out = np.zeros((N, two, I, B))
    for g in range(B // 32):
        byte = sf[:, :, g // 4, :, g % 4, :].reshape(N, two, I).astype(np.int64)
        val = q[..., 32 * g:32 * g + 32].astype(np.float64) * (2.0 ** (byte - 127.0))[..., None]
        out[..., 32 * g:32 * g + 32] = np.where((byte == 255)[..., None], np.nan, val)
    return out


def activation(h, glu="swiglu", interleaved=False, scale=None):
    """a = act(gate) * up of rows h [rows, 2I] (times `scale` per row)."""
    h = np.asarray(h, dtype=np.float64)
    I = h.shape[1] // 2
    g, u = (h[:, 0::2], h[:, 1::2]) if interleaved else (h[:, :I], h[:, I:])
    with np.errstate(over="ignore"):  # e^-g past the range: act = 0
        act = gelu(g) if glu == "geglu" else g / (1 + np.exp(-g))
    a = act * u
    return a if scale is None else a * np.asarray(scale, dtype=np.float64)[:, None]
