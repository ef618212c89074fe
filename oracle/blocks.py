"""Plain fp64 implementations of the operators of include/lstm_blocks.h, written
from their formulas in numpy: the test reference only."""
from __future__ import annotations

import numpy as np


def logistic(x):
    x = np.asarray(x, np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def gated_recurrence(x, forget, input_gate=None, state=None, lengths=None):
    """x, forget, input_gate [B, T, W]; returns (y, state), token by token."""
    B, T, W = x.shape
    y = np.zeros((B, T, W))
    last = np.zeros((B, W)) if state is None else np.array(state, np.float64)
    for b in range(B):
        for t in range(T if lengths is None else int(lengths[b])):
            f = np.asarray(forget[b, t], np.float64)
            w = logistic(-f) if input_gate is None else logistic(input_gate[b, t])
            last[b] = logistic(f) * last[b] + w * x[b, t]
            y[b, t] = last[b]
    return y, last


def gated_recurrence_backward(x, forget, dy, input_gate=None, state=None, dstate=None, lengths=None):
    """Gradients (dx, dforget, dinput_gate, dstate) of gated_recurrence."""
    B, T, W = x.shape
    y, _ = gated_recurrence(x, forget, input_gate, state, lengths)
    dx, df, di = (np.zeros((B, T, W)) for _ in range(3))
    carry = np.zeros((B, W)) if dstate is None else np.array(dstate, np.float64)
    first = np.zeros((B, W)) if state is None else np.asarray(state, np.float64)
    for b in range(B):
        for t in range((T if lengths is None else int(lengths[b])) - 1, -1, -1):
            f = np.asarray(forget[b, t], np.float64)
            a, z = logistic(f), logistic(-f)
            before = y[b, t - 1] if t else first[b]
            D = dy[b, t] + carry[b]
            if input_gate is None:
                dx[b, t], df[b, t] = z * D, D * (before - x[b, t]) * a * z
            else:
                w, v = logistic(input_gate[b, t]), logistic(-np.asarray(input_gate[b, t], np.float64))
                dx[b, t], df[b, t], di[b, t] = w * D, D * before * a * z, D * x[b, t] * w * v
            carry[b] = a * D
    return dx, df, (None if input_gate is None else di), carry


def _turn(u, angle, rot, interleaved, scale, sign=1.0):
    """u [.., heads, D], angle [.., rot / 2]."""
    out = u.copy()
    c, s = scale * np.cos(angle)[..., None, :], sign * scale * np.sin(angle)[..., None, :]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a] = u[..., a] * c - u[..., b] * s
    out[..., b] = u[..., b] * c + u[..., a] * s
    return out


def rotary(x, positions, frequencies, weight=None, norm=False, eps=1e-6, interleaved=False, scale=1.0):
    """x [.., heads, D], positions of its leading axes."""
    u = np.asarray(x, np.float64)
    if norm:
        u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
        if weight is not None:
            u = u * weight
    angle = np.asarray(positions, np.float64)[..., None] * frequencies
    return _turn(u, angle, 2 * len(frequencies), interleaved, scale)


def rotary_backward(x, dy, positions, frequencies, weight=None, norm=False, eps=1e-6, interleaved=False, scale=1.0):
    """Gradients (dx, dweight) of rotary."""
    angle = np.asarray(positions, np.float64)[..., None] * frequencies
    g = _turn(np.asarray(dy, np.float64), angle, 2 * len(frequencies), interleaved, scale, -1.0)
    if not norm:
        return g, None
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    unit = x * r
    dw = (g * unit).reshape(-1, x.shape[-1]).sum(0)
    v = g if weight is None else g * weight
    return r * (v - unit * (v * unit).mean(-1, keepdims=True)), dw


def activation(g, kind):
    """(act(g), its slope)."""
    g = np.asarray(g, np.float64)
    if kind == "gelu":
        k = np.sqrt(2.0 / np.pi)
        t = np.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    p = logistic(g)
    return (p, p * (1 - p)) if kind == "sigmoid" else (g * p, p + g * p * (1 - p))


def gated_mlp(x, w_gate, w_up, w_down, kind):
    """x [rows, in]; returns y."""
    return (activation(x @ w_gate.T, kind)[0] * (x @ w_up.T)) @ w_down.T


def gated_mlp_backward(x, w_gate, w_up, w_down, dy, kind):
    """Gradients (dx, dw_gate, dw_up, dw_down) of gated_mlp."""
    g, u = x @ w_gate.T, x @ w_up.T
    a, slope = activation(g, kind)
    dh = dy @ w_down
    dg, du = dh * u * slope, dh * a
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x, dy.T @ (a * u)
