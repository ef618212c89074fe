"""The operators of include/lstm_ops.h without a GPU: exports, host checks, and
the fp64 oracle's gradients against central differences."""
import ctypes
import os
import re

import numpy as np
import pytest

import layer_lstm_forward_amd as pkg
from layer_lstm_forward_amd import ops
from oracle import ops as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "lstm_ops.h")
FAKE = 0x10000  # never dereferenced: every case below fails a host check first

needs_lib = pytest.mark.skipif(not os.path.exists(pkg.LIB_PATH), reason="liblstm_amd.so not built")


def _shape(**kw):
    a = dict(dtype=1, T=5, B=2, heads=4, kv_heads=2, key_dim=16, value_dim=24, scale=0.25)
    a.update(kw)
    return ops.lstm_linear_attention_shape(**a)


def _v(addr=FAKE):
    return ops.lstm_view(addr, 1, 1, 1)


@needs_lib
def test_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lstm_[a-z_]+)\s*\(", text)))
    assert len(names) == 9
    lib = ctypes.CDLL(pkg.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), f"{n} declared in lstm_ops.h but not exported"
        assert hasattr(ops, n), f"{n} has no binding"


BAD_SHAPES = [(dict(dtype=2), -3), (dict(heads=0), -1), (dict(kv_heads=3), -1), (dict(kv_heads=0), -1),
              (dict(key_dim=0), -1), (dict(key_dim=257), -1), (dict(value_dim=257), -1), (dict(scale=0.0), -1),
              (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(T=0), -2), (dict(B=0), -2),
              (dict(B=1 << 30), -2)]


@needs_lib
@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_linear_attention_shape_checks(kw, code):
    s = _shape(**kw)
    n = ctypes.c_size_t()
    lib = ops._lib()
    assert lib.lstm_linear_attention_workspace_size(s, n) == code
    assert lib.lstm_linear_attention_backward_workspace_size(s, n) == code
    assert ops.lstm_linear_attention_forward(s, _v(), _v(), _v(), FAKE, 0, 0, _v(), 0, FAKE, 1 << 50, 0) == code
    assert ops.lstm_linear_attention_backward(s, _v(), _v(), _v(), FAKE, 0, 0, _v(), 0, _v(), _v(), _v(), 0, FAKE,
                                              1 << 50, 0) == code
    if "T" not in kw:
        s.T = 1
        assert ops.lstm_linear_attention_step(s, _v(), _v(), _v(), FAKE, 0, 99, FAKE, _v(), 0) == code


@needs_lib
def test_linear_attention_argument_checks():
    s, null = _shape(), _v(0)
    for i in range(4):
        a = [_v() for _ in range(4)]
        a[i] = null
        assert ops.lstm_linear_attention_forward(s, a[0], a[1], a[2], FAKE, 0, 0, a[3], 0, FAKE, 1 << 50, 0) == -1
        assert ops.lstm_linear_attention_step(_shape(T=1), a[0], a[1], a[2], FAKE, 0, 99, FAKE, a[3], 0) == -1
    for i in range(7):
        a = [_v() for _ in range(7)]
        a[i] = null
        assert ops.lstm_linear_attention_backward(s, a[0], a[1], a[2], FAKE, 0, 0, a[3], 0, a[4], a[5], a[6], 0,
                                                  FAKE, 1 << 50, 0) == -1
    assert ops.lstm_linear_attention_forward(s, _v(), _v(), _v(), 0, 0, 0, _v(), 0, FAKE, 1 << 50, 0) == -1
    assert ops.lstm_linear_attention_step(s, _v(), _v(), _v(), FAKE, 0, 99, FAKE, _v(), 0) == -2      # T = 5
    one = _shape(T=1)
    assert ops.lstm_linear_attention_step(one, _v(), _v(), _v(), FAKE, 0, 1, FAKE, _v(), 0) == -2     # slots < rows
    assert ops.lstm_linear_attention_step(one, _v(), _v(), _v(), FAKE, FAKE, 0, FAKE, _v(), 0) == -2  # no slots
    assert ops.lstm_linear_attention_step(one, _v(), _v(), _v(), FAKE, 0, 99, 0, _v(), 0) == -1       # no pool
    need = ops.lstm_linear_attention_backward_workspace_size(s)  # shared heads: partial sums
    assert need >= 4 * 5 * 2 * 4 * (16 + 24)
    for ws, size in ((0, 1 << 50), (FAKE, need - 1)):
        assert ops.lstm_linear_attention_backward(s, _v(), _v(), _v(), FAKE, 0, 0, _v(), 0, _v(), _v(), _v(), 0, ws,
                                                  size, 0) == -5
    # good arguments, but no device memory
    assert ops.lstm_linear_attention_backward(s, _v(), _v(), _v(), FAKE, 0, 0, _v(), 0, _v(), _v(), _v(), 0, FAKE,
                                              need, 0) == -4
    assert ops.lstm_linear_attention_step(one, _v(), _v(), _v(), FAKE, 0, 2, FAKE, _v(), 0) == -4


@needs_lib
def test_layer_norm_checks():
    def fwd(dtype=0, x=FAKE, xs=8, res=0, rs=8, rows=3, width=8, eps=1e-5, y=FAKE, sum=0):
        return ops.lstm_layer_norm_forward(dtype, x, xs, res, rs, 0, 0, rows, width, eps, y, sum, 0, 0, 0)

    for kw, code in ((dict(dtype=2), -3), (dict(rows=-1), -2), (dict(width=0), -2), (dict(xs=7), -2),
                     (dict(res=FAKE, rs=7), -2), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
                     (dict(eps=float("inf")), -1), (dict(x=0), -1), (dict(y=0), -1), (dict(sum=FAKE), -1),
                     (dict(rows=0, x=0, y=0), 0), ({}, -4)):
        assert fwd(**kw) == code, kw

    need = ops.lstm_layer_norm_backward_workspace_size(3, 8)
    assert need > 0
    with pytest.raises(pkg.LSTMError):
        ops.lstm_layer_norm_backward_workspace_size(-1, 8)

    def bwd(dtype=0, dy=FAKE, ys=8, z=FAKE, zs=8, mean=FAKE, rstd=FAKE, rows=3, width=8, dx=FAKE, dw=FAKE, ws=FAKE,
            size=need):
        return ops.lstm_layer_norm_backward(dtype, dy, ys, z, zs, mean, rstd, 0, 0, rows, width, dx, dw, 0, ws, size,
                                            0)

    for kw, code in ((dict(dtype=-1), -3), (dict(rows=-1), -2), (dict(width=0), -2), (dict(ys=7), -2),
                     (dict(zs=7), -2), (dict(dy=0), -1), (dict(z=0), -1), (dict(mean=0), -1), (dict(rstd=0), -1),
                     (dict(dx=0), -1), (dict(ws=0), -5), (dict(size=need - 1), -5), ({}, -4)):
        assert bwd(**kw) == code, kw


@needs_lib
def test_adamw_checks():
    def step(dtype=0, bits=32, count=1, b1=0.9, b2=0.99, eps=1e-8, t=1, **kw):
        a = dict(param=FAKE, grad=FAKE, m=FAKE, v=FAKE, n=4, lr=1e-3, weight_decay=0.0)
        a.update(kw)
        tab = (ops.lstm_adamw_tensor * 1)(ops.lstm_adamw_tensor(**a))
        return ops.lstm_adamw_step(dtype, bits, tab, count, b1, b2, eps, t, 0, 0, 0)

    nan = float("nan")
    for kw, code in ((dict(dtype=2), -3), (dict(bits=16), -7), (dict(count=-1), -1), (dict(b1=1.0), -1),
                     (dict(b1=-0.1), -1), (dict(b2=nan), -1), (dict(eps=-1.0), -1), (dict(t=0), -1), (dict(n=-1), -2),
                     (dict(lr=nan), -1), (dict(weight_decay=nan), -1), (dict(param=0), -1), (dict(grad=0), -1),
                     (dict(m=0), -1), (dict(v=0), -1), (dict(bits=8), -1), (dict(master=FAKE), -1), ({}, -4)):
        assert step(**kw) == code, kw
    assert ops.lstm_adamw_step(0, 32, None, 1, 0.9, 0.99, 1e-8, 1, 0, 0, 0) == -1


def test_wrappers_refuse_host_tensors():
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        pkg.layer_norm(x)
    q = torch.zeros(3, 2, 4, 8)
    with pytest.raises(ValueError):
        pkg.linear_attention(q, q, q, torch.zeros(4))
    with pytest.raises(ValueError):
        pkg.adamw_step([x], [x], [x], [x], step=1)


# ----------------------------------------------- the oracle's own gradients
def _differences(f, x, at, h=1e-5):
    out = []
    for i in at:
        d = np.zeros(x.size)
        d[i] = h
        d = d.reshape(x.shape)
        out.append((f(x + d) - f(x - d)) / (2 * h))
    return np.array(out)


def test_oracle_linear_attention_gradients_are_differences():
    rng = np.random.default_rng(3)
    B, T, H, G, Dk, Dv = 2, 6, 4, 2, 3, 5
    q, k, v = rng.normal(size=(B, T, H, Dk)), rng.normal(size=(B, T, G, Dk)), rng.normal(size=(B, T, G, Dv))
    S, do, dS = rng.normal(size=(B, H, Dk, Dv)), rng.normal(size=(B, T, H, Dv)), rng.normal(size=(B, H, Dk, Dv))
    g, n = np.log([0.5, 0.9, 0.99, 1.0]), [6, 4]

    def loss(q, k, v, S):
        o, last = ref.linear_attention(q, k, v, g, 0.7, S, n)
        return (o * do).sum() + (last * dS).sum()

    grads = ref.linear_attention_backward(q, k, v, g, 0.7, do, S, dS, n)
    args = [q, k, v, S]
    for i, got in enumerate(grads):
        at = rng.choice(args[i].size, 12, replace=False)
        want = _differences(lambda x: loss(*args[:i], x, *args[i + 1:]), args[i], at)
        # central differences of a polynomial of degree at most 3 in one entry: rounding of the loss only
        np.testing.assert_allclose(got.reshape(-1)[at], want, rtol=0, atol=1e-6)


def test_oracle_layer_norm_gradients_are_differences():
    rng = np.random.default_rng(4)
    z, dy, ds = (rng.normal(size=(3, 7)) for _ in range(3))
    w, b = rng.normal(size=7), rng.normal(size=7)

    def loss(z, w, b):
        return (ref.layer_norm(z, w, b)[0] * dy).sum() + (z * ds).sum()

    dz, dw, db = ref.layer_norm_backward(dy, z, w, dsum=ds)
    args = [z, w, b]
    for i, got in enumerate((dz, dw, db)):
        want = _differences(lambda x: loss(*args[:i], x, *args[i + 1:]), args[i], range(args[i].size))
        np.testing.assert_allclose(got.reshape(-1), want, rtol=0, atol=1e-6)


@needs_lib
def test_limits():
    assert ops.lstm_layer_norm_forward(0, FAKE, 1 << 30, 0, 0, 0, 0, 1, (1 << 28) + 1, 1e-5, FAKE, 0, 0, 0, 0) == -2
    # steps from token to token are 32-bit byte counts
    far = ops.lstm_view(FAKE, 1 << 30, 1, 1)
    assert ops.lstm_linear_attention_forward(_shape(), far, _v(), _v(), FAKE, 0, 0, _v(), 0, FAKE, 1 << 50, 0) == -2
    assert ops.lstm_linear_attention_backward(_shape(), _v(), _v(), far, FAKE, 0, 0, _v(), 0, _v(), _v(), _v(), 0, FAKE,
                                              1 << 50, 0) == -2
