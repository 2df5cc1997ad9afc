"""Float64 oracle of the gated feed-forward block, forward and backward: h = x W1 + b1, a = act(gate) up, out = a W2 + b2.
Columns of W1, b1 and h: gate then up, or interleaved (gate_i at 2i, up_i at 2i + 1)."""
import numpy as np
from scipy.special import erf


def split(h, interleaved):
    I = h.shape[-1] // 2
    return (h[..., 0::2], h[..., 1::2]) if interleaved else (h[..., :I], h[..., I:])


def join(gate, up, interleaved):
    if not interleaved:
        return np.concatenate([gate, up], -1)
    out = np.empty(gate.shape[:-1] + (2 * gate.shape[-1],))
    out[..., 0::2], out[..., 1::2] = gate, up
    return out


def activation(g, gelu):
    """act(g) and act'(g)."""
    if gelu:
        cdf = 0.5 * (1 + erf(g / np.sqrt(2)))
        return g * cdf, cdf + g * np.exp(-0.5 * g * g) / np.sqrt(2 * np.pi)
    s = 0.5 * (1 + np.tanh(0.5 * g))
    return g * s, s * (1 + g * (1 - s))


def forward(x, W1, W2, b1=None, b2=None, gelu=False, interleaved=False):
    """out and h."""
    h = x @ W1 + (0 if b1 is None else b1)
    gate, up = split(h, interleaved)
    return (activation(gate, gelu)[0] * up) @ W2 + (0 if b2 is None else b2), h


def backward(dout, x, h, W1, W2, gelu=False, interleaved=False):
    """dx, dW1, dW2, db1, db2, and the intermediate da, dh and a."""
    gate, up = split(h, interleaved)
    act, slope = activation(gate, gelu)
    da = dout @ W2.T
    dh = join(da * up * slope, da * act, interleaved)
    a = act * up
    return dict(dx=dh @ W1.T, dW1=x.T @ dh, dW2=a.T @ dout, db1=dh.sum(0), db2=dout.sum(0), da=da, dh=dh, a=a)
