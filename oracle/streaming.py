"""Plain NumPy definition of the streaming-block operators (oracle).

TEST INFRASTRUCTURE ONLY -- see the package docstring.  One sequence (or one
row) at a time in fp64, written from the formulas in the header: the INT4-g64
linear layer, the causal depthwise convolution with a state, the selective
state-space scan and the residual update with the norms around it.
"""
from __future__ import annotations

import numpy as np

__all__ = ["unpack_int4", "quant_linear", "causal_conv", "scan_clip", "op_activation", "op_norm", "residual_norm"]


def op_activation(v, act):
    if act == "swish":
        return v / (1.0 + np.exp(-v))
    if act == "sigmoid":
        return 1.0 / (1.0 + np.exp(-v))
    return np.tanh(v) if act == "tanh" else v


def unpack_int4(packed: np.ndarray) -> np.ndarray:
    """uint8 [n, k / 2] -> integers [n, k]: in each little-endian 32-bit word weight
    2 i sits in bits 4 i .. and weight 2 i + 1 in bits 16 + 4 i .., stored plus 8."""
    words = np.ascontiguousarray(packed).view("<u4").astype(np.int64)
    q = np.empty(words.shape + (8,), np.int64)
    for i in range(4):
        q[..., 2 * i] = (words // 16 ** i) % 16 - 8
        q[..., 2 * i + 1] = (words // 16 ** (4 + i)) % 16 - 8
    return q.reshape(words.shape[0], -1)


def quant_linear(x, q, scale, bias=None, act="none"):
    """x [rows, k], q integers [n, k], scale [n, k / 64]."""
    w = q.astype(np.float64) * np.repeat(scale.astype(np.float64), 64, axis=1)
    y = x.astype(np.float64) @ w.T
    return op_activation(y if bias is None else y + bias, act)


def causal_conv(x, w, bias=None, state=None, act="none"):
    """x [t, d], w [d, taps], state [taps - 1, d] -> (y [t, d], new state)."""
    d, taps = w.shape
    past = np.zeros((taps - 1, d)) if state is None else state.astype(np.float64)
    v = np.concatenate([past, x.astype(np.float64)])
    y = np.zeros((len(x), d))
    for t in range(len(x)):
        for j in range(taps):
            y[t] += w[:, j] * v[t + j]
    return op_activation(y if bias is None else y + bias, act), v[len(x):]


def scan_clip(x, dt, a, b, c, d_skip=None, z=None, dt_bias=None, softplus=True, state=None):
    """x, dt, z [t, d], a [d, n], b, c [t, n], state [d, n] -> (y [t, d], new state, E)
    where E [t, d] bounds |error of y| before the gate of an fp32 evaluation:

    With u = 2^-24, the step s carries <= 8 u (bias add, exp, log1p, rounding of
    dt's type is exact), the exponent s a log2(e) three more roundings, so the
    decay e is off by <= (|s a| 11 u + 4 u) e (the hardware's exp2 is within 2
    steps, 4 u), and the input s x b by <= 10 u of itself.  A frame's update adds
    one rounding of h.  The error bound of h obeys the recurrence itself:
    E' = e (1 + delta) E + delta e |h| + 10 u |s x b| + u |h'|.  y adds a sum of n
    products and the skip term, <= (n + 4) u of the terms' magnitudes.  The bound
    of an evaluation in two pieces joined over a frame axis is at most twice it."""
    u = 2.0 ** -24
    f = np.float64
    x, dt, a, b, c = (np.asarray(v, f) for v in (x, dt, a, b, c))
    t, d = x.shape
    h = np.zeros(a.shape) if state is None else np.asarray(state, f).copy()
    eh = np.zeros_like(h)
    y, ey = np.zeros((t, d)), np.zeros((t, d))
    skip = np.zeros(d) if d_skip is None else np.asarray(d_skip, f)
    for i in range(t):
        raw = dt[i] if dt_bias is None else dt[i] + dt_bias
        s = np.logaddexp(0, raw) if softplus else raw
        # a cancelling sum dt + bias is off by u of its terms, and so is what softplus makes of it
        ds = 8 * u * np.abs(s) + u * (np.abs(dt[i]) + np.abs(raw)) * (np.abs(s) if softplus else 1)
        e = np.exp(s[:, None] * a)
        delta = np.abs(a) * ds[:, None] + 4 * u * np.abs(s[:, None] * a) + 4 * u
        inc = (s * x[i])[:, None] * b[i]
        dinc = np.abs(x[i] * ds)[:, None] * np.abs(b[i]) + 2 * u * np.abs(inc)
        new = e * h + inc
        eh = e * (1 + delta) * eh + delta * e * np.abs(h) + dinc + 2 * u * np.abs(new) + 2.0 ** -120
        h = new
        y[i] = h @ c[i] + skip * x[i]
        ey[i] = eh @ np.abs(c[i]) + (a.shape[1] + 4) * u * (np.abs(h) @ np.abs(c[i]) + np.abs(skip * x[i]))
    if z is not None:
        g = op_activation(np.asarray(z, f), "swish")
        y, ey = y * g, ey * np.abs(g) + 8 * u * np.abs(y * g)
    return y, h, ey, eh


def op_norm(v, kind, weight=None, bias=None, eps=1e-5):
    if kind == "layer":
        v = v - v.mean()
    if kind != "none":
        v = v / np.sqrt((v * v).mean() + eps)
        v = v if weight is None else v * weight
    return v + bias if kind == "layer" and bias is not None else v


def residual_norm(x, y, alpha=1.0, layer_scale=None, gate=None, gate_act="none", post="none", post_weight=None,
                  post_bias=None, pre="layer", pre_weight=None, pre_bias=None, eps=1e-5):
    """One row: x, y [d], gate [d] or None -> (x', u)."""
    br = alpha * op_norm(y, post, post_weight, post_bias, eps)
    if gate is not None:
        br = br * op_activation(gate, gate_act)
    if layer_scale is not None:
        br = br * layer_scale
    x = x + br
    return x, op_norm(x, pre, pre_weight, pre_bias, eps)
