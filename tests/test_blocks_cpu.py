"""The operators of include/lstm_blocks.h without a GPU: exports, host checks,
the fp64 oracle's gradients against central differences, and the wrappers'
refusals and use of streams."""
import ctypes
import os
import re

import numpy as np
import pytest

import layer_lstm_forward_amd as pkg
from layer_lstm_forward_amd import block_ops as ops
from layer_lstm_forward_amd.ops import lstm_view
from oracle import blocks as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "lstm_blocks.h")
FAKE = 0x10000  # never dereferenced: every case below fails a host check first

needs_lib = pytest.mark.skipif(not os.path.exists(pkg.LIB_PATH), reason="liblstm_amd.so not built")


def _v(addr=FAKE):
    return lstm_view(addr, 1, 1, 1)


@needs_lib
def test_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lstm_[a-z_]+)\s*\(", text)))
    assert len(names) == 13
    lib = ctypes.CDLL(pkg.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), f"{n} declared in lstm_blocks.h but not exported"
        assert hasattr(ops, n), f"{n} has no binding"


def _rec(**kw):
    return ops.lstm_gated_recurrence_shape(**{**dict(dtype=1, T=5, B=2, width=16), **kw})


@needs_lib
@pytest.mark.parametrize("kw,code", [(dict(dtype=2), -3), (dict(T=0), -2), (dict(T=(1 << 30) + 1), -2), (dict(B=0), -2),
                                     (dict(width=0), -2), (dict(width=(1 << 20) + 1), -2),
                                     (dict(B=1 << 20, width=1 << 11), -2), (None, -1)])
def test_recurrence_shape_checks(kw, code):
    s = None if kw is None else _rec(**kw)
    n = ctypes.c_size_t()
    lib = ops._lib()
    assert lib.lstm_gated_recurrence_workspace_size(s, n) == code
    assert lib.lstm_gated_recurrence_backward_workspace_size(s, n) == code
    assert ops.lstm_gated_recurrence_forward(s, _v(), _v(), None, 0, 0, _v(), 0, FAKE, 1 << 50, 0) == code
    assert ops.lstm_gated_recurrence_backward(s, _v(), _v(), None, 0, 0, _v(), _v(), 0, _v(), _v(), None, 0, FAKE,
                                              1 << 50, 0) == code
    if kw is None or "T" not in kw:
        if s is not None:
            s.T = 1
        assert ops.lstm_gated_recurrence_step(s, _v(), _v(), None, 0, 99, FAKE, _v(), 0) == code


@needs_lib
def test_recurrence_argument_checks():
    s, null, one = _rec(), _v(0), _rec(T=1)
    fwd = lambda s, a, ws=FAKE, size=1 << 50: ops.lstm_gated_recurrence_forward(  # noqa: E731
        s, a[0], a[1], a[2], 0, 0, a[3], 0, ws, size, 0)
    for bad in (null, None):
        for i in (0, 1, 3):
            a = [_v(), _v(), None, _v()]
            a[i] = bad
            assert fwd(s, a) == -1
            assert ops.lstm_gated_recurrence_step(one, a[0], a[1], a[2], 0, 9, FAKE, a[3], 0) == -1
    assert fwd(s, [_v(), _v(), null, _v()]) == -1  # an input gate without memory
    for i in range(6):
        a = [_v() for _ in range(6)]
        a[i] = null
        assert ops.lstm_gated_recurrence_backward(s, a[0], a[1], None, 0, 0, a[2], a[3], 0, a[4], a[5], None, 0, FAKE,
                                                  1 << 50, 0) == -1
    for i, di in ((_v(), None), (None, _v()), (_v(), null)):  # the input gate's gradient goes with the gate
        assert ops.lstm_gated_recurrence_backward(s, _v(), _v(), i, 0, 0, _v(), _v(), 0, _v(), _v(), di, 0, FAKE,
                                                  1 << 50, 0) == -1
    long = _rec(T=4096, B=1)
    need = ops.lstm_gated_recurrence_workspace_size(long)
    assert need > 0
    for ws, size in ((0, 1 << 50), (FAKE, need - 1)):
        assert fwd(long, [_v(), _v(), None, _v()], ws, size) == -5
    assert ops.lstm_gated_recurrence_step(s, _v(), _v(), None, 0, 9, FAKE, _v(), 0) == -2       # T = 5
    assert ops.lstm_gated_recurrence_step(one, _v(), _v(), None, 0, 1, FAKE, _v(), 0) == -2     # slots < rows
    assert ops.lstm_gated_recurrence_step(one, _v(), _v(), None, FAKE, 0, FAKE, _v(), 0) == -2  # no slots
    assert ops.lstm_gated_recurrence_step(one, _v(), _v(), None, 0, 9, 0, _v(), 0) == -1        # no pool
    assert fwd(s, [_v(), _v(), _v(), _v()]) == -4  # good arguments, but no device memory


@needs_lib
@pytest.mark.parametrize("dtype", [0, 1])
def test_recurrence_workspace_alignment(dtype):
    """Where the workspace holds words that travel whole, it is taken at its alignment or refused."""
    s = _rec(T=4096, B=1, dtype=dtype)
    for off, code in ((8, -1), (4, -1), (1, -1), (16, -4)):  # the last: good arguments, but no device memory
        assert ops.lstm_gated_recurrence_forward(s, _v(), _v(), None, 0, 0, _v(), 0, FAKE + off, 1 << 50, 0) == code
        assert ops.lstm_gated_recurrence_backward(s, _v(), _v(), None, 0, 0, _v(), _v(), 0, _v(), _v(), None, 0,
                                                  FAKE + off, 1 << 50, 0) == code


def _rot(**kw):
    return ops.lstm_rotary_shape(**{**dict(dtype=0, T=5, B=2, heads=4, kv_heads=2, dim=16, rotary_dim=8, interleaved=0,
                                           norm=1, eps=1e-6, scale=1.0), **kw})


@needs_lib
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), -3), (dict(heads=0), -1), (dict(heads=65537), -1), (dict(kv_heads=-1), -1), (dict(dim=0), -1),
    (dict(dim=257), -1), (dict(rotary_dim=7), -1), (dict(rotary_dim=18), -1), (dict(rotary_dim=-2), -1),
    (dict(interleaved=2), -1), (dict(norm=-1), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(scale=float("inf")), -1), (dict(T=0), -2), (dict(B=0), -2),
    (dict(T=1 << 16, B=1 << 15), -2), (None, -1)])
def test_rotary_shape_checks(kw, code):
    s = None if kw is None else _rot(**kw)
    assert ops._lib().lstm_rotary_backward_workspace_size(s, ctypes.c_size_t()) == code
    assert ops.lstm_rotary_forward(s, _v(), _v(), 0, 0, FAKE, None, _v(), _v(), 0) == code
    assert ops.lstm_rotary_backward(s, _v(), _v(), 0, 0, FAKE, None, _v(), _v(), _v(), _v(), 0, 0, FAKE, 1 << 50,
                                    0) == code


@needs_lib
def test_rotary_argument_checks():
    null = _v(0)

    def fwd(s, q=_v(), k=_v(), wq=0, wk=0, f=FAKE, qo=_v(), ko=_v()):
        return ops.lstm_rotary_forward(s, q, k, wq, wk, f, None, qo, ko, 0)

    def bwd(s, q=_v(), k=_v(), wq=0, wk=0, f=FAKE, dqo=_v(), dko=_v(), dq=_v(), dk=_v(), dwq=0, dwk=0, ws=FAKE,
            size=1 << 50):
        return ops.lstm_rotary_backward(s, q, k, wq, wk, f, None, dqo, dko, dq, dk, dwq, dwk, ws, size, 0)

    for n in ("q", "k", "qo", "ko"):
        assert fwd(_rot(), **{n: null}) == -1 and fwd(_rot(), **{n: None}) == -1
    for n in ("q", "k", "dqo", "dko", "dq", "dk"):
        assert bwd(_rot(), **{n: null}) == -1
    alone = _rot(kv_heads=0)
    assert fwd(alone, k=None, ko=None) == -4 and bwd(alone, k=None, dko=None, dk=None) == -4
    plain = _rot(norm=0)
    assert fwd(plain, wq=FAKE) == -1 and fwd(plain, wk=FAKE) == -1
    for n in ("wq", "wk", "dwq", "dwk"):
        assert bwd(plain, **{n: FAKE}) == -1
    assert bwd(plain, q=None, k=None) == -4  # without a norm the inputs are not read
    assert fwd(_rot(), f=0) == -1 and bwd(_rot(), f=0) == -1 and fwd(_rot(rotary_dim=0), f=0) == -4
    need = ops.lstm_rotary_backward_workspace_size(_rot())
    assert need > 0 and ops.lstm_rotary_backward_workspace_size(plain) == 0
    assert bwd(_rot(), dwq=FAKE, ws=0) == -5 and bwd(_rot(), dwk=FAKE, size=need - 1) == -5
    assert bwd(_rot(), ws=0) == -4  # no sums wanted: no workspace


def _mlp(**kw):
    a = {**dict(dtype=1, activation=0, rows=4, hidden=24, out=16), **{k: v for k, v in kw.items() if k != "width"}}
    s = ops.lstm_gated_mlp_shape(**a)
    setattr(s, "in", kw.get("width", 8))
    return s


@needs_lib
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -3), (dict(activation=3), -1), (dict(activation=-1), -1), (dict(rows=-1), -2), (dict(width=0), -2),
    (dict(hidden=0), -2), (dict(out=0), -2), (dict(width=(1 << 18) + 1), -2), (dict(hidden=(1 << 18) + 1), -2),
    (dict(out=(1 << 18) + 1), -2), (dict(rows=1 << 21, hidden=1 << 18), -2), (dict(rows=(1 << 30) + 1), -2),
    (None, -1)])
def test_mlp_shape_checks(kw, code):
    s = None if kw is None else _mlp(**kw)
    n, lib, big = ctypes.c_size_t(), ops._lib(), 1 << 50
    for f in (lib.lstm_gated_mlp_workspace_size, lib.lstm_gated_mlp_reserve_size,
              lib.lstm_gated_mlp_backward_workspace_size):
        assert f(s, n) == code
    assert ops.lstm_gated_mlp_forward(s, FAKE, 1 << 20, FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, big, 0) == code
    assert ops.lstm_gated_mlp_backward(s, FAKE, 1 << 20, FAKE, FAKE, FAKE, FAKE, big, FAKE, 1 << 20, FAKE, FAKE, FAKE,
                                       FAKE, FAKE, big, 0) == code


@needs_lib
def test_mlp_argument_checks():
    s, big = _mlp(), 1 << 50

    def fwd(s=s, x=FAKE, xs=8, g=FAKE, u=FAKE, d=FAKE, y=FAKE, r=0, rb=0, ws=FAKE, size=big):
        return ops.lstm_gated_mlp_forward(s, x, xs, g, u, d, y, r, rb, ws, size, 0)

    def bwd(s=s, x=FAKE, xs=8, g=FAKE, u=FAKE, d=FAKE, r=FAKE, rb=big, dy=FAKE, ys=16, ws=FAKE, size=big):
        return ops.lstm_gated_mlp_backward(s, x, xs, g, u, d, r, rb, dy, ys, FAKE, FAKE, FAKE, FAKE, ws, size, 0)

    need, back = ops.lstm_gated_mlp_workspace_size(s), ops.lstm_gated_mlp_backward_workspace_size(s)
    held = ops.lstm_gated_mlp_reserve_size(s)
    for kw, code in ((dict(xs=7), -2), (dict(x=0), -1), (dict(g=0), -1), (dict(u=0), -1), (dict(d=0), -1),
                     (dict(y=0), -1), (dict(g=FAKE + 8), -1), (dict(u=FAKE + 2), -1), (dict(d=FAKE + 4), -1),
                     (dict(ws=FAKE + 8), -1), (dict(r=FAKE + 8, rb=big), -1), (dict(ws=0), -5),
                     (dict(size=need - 1), -5), (dict(r=FAKE, rb=held - 1), -5), ({}, -4), (dict(r=FAKE, rb=held), -4),
                     (dict(s=_mlp(rows=0), x=0, y=0, ws=0, size=0), 0)):
        assert fwd(**kw) == code, kw
    for kw, code in ((dict(xs=7), -2), (dict(ys=15), -2), (dict(x=0), -1), (dict(g=0), -1), (dict(u=0), -1),
                     (dict(d=0), -1), (dict(r=0), -1), (dict(dy=0), -1), (dict(d=FAKE + 8), -1),
                     (dict(r=FAKE + 8), -1), (dict(rb=held - 1), -5), (dict(ws=0), -5), (dict(size=back - 1), -5),
                     ({}, -4)):
        assert bwd(**kw) == code, kw


def _slopes(f, args, grads, cotangent, h=1e-6):
    """Every gradient against central differences of <f(args), cotangent>."""
    for k, (a, g) in enumerate(zip(args, grads)):
        if a is None:
            continue
        d = np.zeros(a.shape)
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = f(*args)
            a[i] = keep - h
            down = f(*args)
            a[i] = keep
            d[i] = sum(((u - v) * c).sum() for u, v, c in zip(up, down, cotangent)) / (2 * h)
        assert np.allclose(d, g, rtol=1e-6, atol=1e-7), k


@pytest.mark.parametrize("gates", [1, 2])
def test_recurrence_oracle_gradients(gates):
    rng = np.random.default_rng(1)
    B, T, W = 2, 4, 3
    x, f, dy = (rng.standard_normal((B, T, W)) for _ in range(3))
    i = rng.standard_normal((B, T, W)) if gates == 2 else None
    S, dS = rng.standard_normal((2, B, W))
    run = lambda x, f, i, S: ref.gated_recurrence(x, f, i, S, [4, 2])  # noqa: E731
    dx, df, di, ds = ref.gated_recurrence_backward(x, f, dy, i, S, dS, [4, 2])
    _slopes(run, [x, f, i, S], [dx, df, di, ds], [dy, dS])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary_oracle_gradients(norm, interleaved):
    rng = np.random.default_rng(2)
    x, dy, w = rng.standard_normal((3, 2, 7)), rng.standard_normal((3, 2, 7)), rng.standard_normal(7)
    pos, f = np.array([0, 5, -3]), np.array([1.0, 0.3])
    more = dict(norm=norm, eps=0.01, interleaved=interleaved, scale=1.3)
    dx, dw = ref.rotary_backward(x, dy, pos, f, w if norm else None, **more)
    _slopes(lambda x, w: [ref.rotary(x, pos, f, w, **more)], [x, w if norm else None], [dx, dw], [dy])
    # a turn keeps lengths, and undoes itself
    y = ref.rotary(x, pos, f, interleaved=interleaved)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose(ref.rotary(y, -pos, f, interleaved=interleaved), x)


@pytest.mark.parametrize("kind", ["silu", "gelu", "sigmoid"])
def test_mlp_oracle_gradients(kind):
    rng = np.random.default_rng(3)
    x, wg, wu, wd, dy = (rng.standard_normal(s) for s in ((3, 4), (5, 4), (5, 4), (2, 5), (3, 2)))
    grads = ref.gated_mlp_backward(x, wg, wu, wd, dy, kind)
    _slopes(lambda *a: [ref.gated_mlp(*a, kind)], [x, wg, wu, wd], grads, [dy])


# ------------------------------------------------------------- the wrappers
from tests.test_ops_streams_cpu import MAIN, NOTES, SIDE, check, device, put  # noqa: E402,F401  (device: a fixture)


@pytest.fixture
def kernels(monkeypatch):
    from tests import test_ops_streams_cpu as streams
    make = streams.torch.Tensor.new_empty
    monkeypatch.setattr(streams.Device, "new_empty",
                        lambda t, *a: NOTES.append(("allocation", streams.NOW[0])) or make(t, *a), raising=False)
    for name in dir(ops):
        if name.startswith("lstm_") and callable(getattr(ops, name)) and not isinstance(getattr(ops, name), type):
            size = name.endswith("_size")
            monkeypatch.setattr(ops, name, (lambda *a: 64) if size else lambda *a: NOTES.append(("kernels", a[-1])) or 0)


def test_streams(kernels):
    x, S = put(5, 2, 8), put(2, 8)
    y, _ = pkg.gated_recurrence(x, x, lengths=[5, 2], stream=SIDE)
    check(0, 2)
    pkg.gated_recurrence_backward(x, x, y, x, input_gate=x, state=S, lengths=[5, 2], stream=SIDE)
    check(0, 4)
    pkg.gated_recurrence_step(x[0], x[0], S, stream=SIDE)
    check(0, 1)
    import torch
    q, f = put(5, 2, 4, 8), torch.zeros(4, dtype=torch.float64).as_subclass(type(x))
    a, b = pkg.rotary(q, q, f, stream=SIDE)
    check(0, 2)
    pkg.rotary_backward(q, q, f, a, b, norm=True, stream=SIDE)
    check(0, 4)
    w, wd, t = put(6, 8), put(3, 6), put(4, 3, 8).transpose(0, 1)
    y, kept = pkg.gated_mlp_train(t, w, w, wd, stream=SIDE)
    check(1, 2)
    pkg.gated_mlp_backward(y.transpose(0, 1).contiguous().transpose(0, 1), t, w, w, wd, kept, stream=SIDE)
    NOTES.remove(("copy", MAIN))
    check(2, 4)
    pkg.gated_mlp(t, w, w, wd)  # the current stream: no switch, nothing to give
    assert set(NOTES) == {("copy", MAIN), ("allocation", MAIN), ("kernels", MAIN)}


def test_refusals(kernels):
    import torch
    x, S = put(5, 2, 8), put(2, 8)
    D = type(x)
    half, f = x.half().as_subclass(D), torch.zeros(4, dtype=torch.float64).as_subclass(D)
    q, w, wd = put(5, 2, 4, 8), put(6, 8), put(3, 6)
    pos = torch.zeros(5, 2, dtype=torch.int32).as_subclass(D)
    kept = torch.zeros(64, dtype=torch.uint8).as_subclass(D)
    for call in (
            lambda: pkg.gated_recurrence(half, half), lambda: pkg.gated_recurrence(x[0], x[0]),
            lambda: pkg.gated_recurrence(x, x[:4]), lambda: pkg.gated_recurrence(x, half),
            lambda: pkg.gated_recurrence(put(5, 8, 2).transpose(1, 2), x), lambda: pkg.gated_recurrence(x, x, x[:, :1]),
            lambda: pkg.gated_recurrence(x, x, state=S[:1]), lambda: pkg.gated_recurrence(x, x, state=S.double()),
            lambda: pkg.gated_recurrence(x, x, lengths=[6, 0]), lambda: pkg.gated_recurrence(x, x, lengths=[1]),
            lambda: pkg.gated_recurrence(x, x, out=(x[:4], S)),
            lambda: pkg.gated_recurrence_backward(x, x, x[:4], x), lambda: pkg.gated_recurrence_backward(x, x, x, half),
            lambda: pkg.gated_recurrence_backward(x, x, x, x, dstate=S[:1]),
            lambda: pkg.gated_recurrence_backward(x, x, x, x, out=(x, x, x)),
            lambda: pkg.gated_recurrence_step(x, x, S), lambda: pkg.gated_recurrence_step(x[0], x[0], S[:, :4]),
            lambda: pkg.gated_recurrence_step(x[0], x[0], S, slots=torch.zeros(2).as_subclass(D)),
            lambda: pkg.rotary(half, None, f), lambda: pkg.rotary(q[0, 0], None, f), lambda: pkg.rotary(q, q[0], f),
            lambda: pkg.rotary(q, q[:, :1], f), lambda: pkg.rotary(q, q[..., :4], f),
            lambda: pkg.rotary(q, q, f.float()), lambda: pkg.rotary(q, q, f[None]),
            lambda: pkg.rotary(q, q, f, positions=pos.long()), lambda: pkg.rotary(q, q, f, positions=pos[:4]),
            lambda: pkg.rotary(q, q, f, q_weight=put(8)), lambda: pkg.rotary(q, q, f, q_weight=put(7), norm=True),
            lambda: pkg.rotary(q, q, f, out=(q, q[:4])), lambda: pkg.rotary_backward(q, q, f, q[:4], q),
            lambda: pkg.rotary_backward(q, q, f, q, q[:4]), lambda: pkg.rotary_frequencies(7, device="cpu"),
            lambda: pkg.rotary_frequencies(8, base=0, device="cpu"),
            lambda: pkg.rotary_frequencies(8, factor=-1, device="cpu"),
            lambda: pkg.rotary_frequencies(8, original_length=100, low=4, high=4, device="cpu"),
            lambda: pkg.gated_mlp(half, w, w, wd), lambda: pkg.gated_mlp(x, w, w, wd, activation="relu"),
            lambda: pkg.gated_mlp(x, w, put(7, 8), wd), lambda: pkg.gated_mlp(x, w, w, put(3, 7)),
            lambda: pkg.gated_mlp(x, put(8, 6).T, w, wd), lambda: pkg.gated_mlp(x, w[0], w, wd),
            lambda: pkg.gated_mlp(put(4, 7), w, w, wd), lambda: pkg.gated_mlp(put(4, 0), w, w, wd),
            lambda: pkg.gated_mlp_backward(x, x, w, w, wd, kept),
            lambda: pkg.gated_mlp_backward(put(5, 2, 3), x, w, w, wd, kept[:8])):
        with pytest.raises(ValueError):
            call()
    assert not [n for n in NOTES if n[0] == "kernels"]


def test_refuses_a_reserve_with_gaps(kernels):
    import torch
    x, w, wd = put(5, 2, 8), put(6, 8), put(3, 6)
    wide = torch.zeros(128, dtype=torch.uint8).as_subclass(type(x))
    with pytest.raises(ValueError):
        pkg.gated_mlp_backward(put(5, 2, 3), x, w, w, wd, wide[::2])
    assert not [n for n in NOTES if n[0] == "kernels"]
    pkg.gated_mlp_backward(put(5, 2, 3), x, w, w, wd, wide[:64])
