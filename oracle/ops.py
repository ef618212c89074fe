"""Plain fp64 implementations of the operators of include/lstm_ops.h, written
from their formulas in numpy: the test reference only."""
from __future__ import annotations

import numpy as np


def linear_attention(q, k, v, log_decay, scale, state=None, lengths=None):
    """q [B, T, H, Dk], k [B, T, G, Dk], v [B, T, G, Dv]; returns (o, state), token by token."""
    B, T, H, Dk = q.shape
    G, Dv = k.shape[2], v.shape[3]
    share = np.arange(H) // (H // G)
    gamma = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    o = np.zeros((B, T, H, Dv))
    last = np.zeros((B, H, Dk, Dv)) if state is None else np.array(state, np.float64)
    for b in range(B):
        S = last[b]
        for t in range(T if lengths is None else int(lengths[b])):
            S = gamma * S + k[b, t, share][:, :, None] * v[b, t, share][:, None, :]
            o[b, t] = scale * np.einsum("hd,hde->he", q[b, t], S)
        last[b] = S
    return o, last


def linear_attention_backward(q, k, v, log_decay, scale, do, state=None, dstate=None, lengths=None):
    """Gradients (dq, dk, dv, dstate) of linear_attention: the recurrence backwards, token by token."""
    B, T, H, Dk = q.shape
    G, Dv = k.shape[2], v.shape[3]
    per = H // G
    share = np.arange(H) // per
    gamma = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    dq, dk, dv = (np.zeros(x.shape) for x in (q, k, v))
    first = np.zeros((B, H, Dk, Dv))
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        S = np.zeros((H, Dk, Dv)) if state is None else np.array(state[b], np.float64)
        for t in range(n):
            S = gamma * S + k[b, t, share][:, :, None] * v[b, t, share][:, None, :]
            dq[b, t] = scale * np.einsum("hde,he->hd", S, do[b, t])
        D = np.zeros((H, Dk, Dv)) if dstate is None else np.array(dstate[b], np.float64)
        for t in range(n - 1, -1, -1):
            D = D + scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            dk[b, t] = np.einsum("hde,he->hd", D, v[b, t, share]).reshape(G, per, Dk).sum(1)
            dv[b, t] = np.einsum("hde,hd->he", D, k[b, t, share]).reshape(G, per, Dv).sum(1)
            D = gamma * D
        first[b] = D
    return dq, dk, dv, first


def layer_norm(z, weight=None, bias=None, eps=1e-5):
    """Over the rows of z [rows, width]; returns (y, mean, rstd)."""
    z = np.asarray(z, np.float64)
    mean = z.sum(1) / z.shape[1]
    rstd = 1.0 / np.sqrt(((z - mean[:, None]) ** 2).sum(1) / z.shape[1] + eps)
    y = (z - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_backward(dy, z, weight=None, eps=1e-5, dsum=None):
    """Gradients (dz, dweight, dbias) of layer_norm."""
    z, dy = np.asarray(z, np.float64), np.asarray(dy, np.float64)
    unit, _, rstd = layer_norm(z, eps=eps)
    g = dy if weight is None else dy * weight
    n = z.shape[1]
    dz = rstd[:, None] * (g - g.sum(1, keepdims=True) / n - unit * (g * unit).sum(1, keepdims=True) / n)
    return (dz if dsum is None else dz + dsum), (dy * unit).sum(0), dy.sum(0)


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay):
    """One step; returns (p, m, v)."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    hat = (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - lr * hat, m, v


def code_values():
    """The value of every 8-bit code (4 exponent bits of bias 7, 3 fraction bits; 0x7F and 0xFF are not numbers)."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e > 0, 2.0 ** (e - 7) * (1 + f / 8), f * 2.0 ** -9)
    x = np.where(c & 127 == 127, np.nan, x)
    return np.where(c >= 128, -x, x)
