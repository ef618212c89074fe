"""Which stream the wrappers' own copies and allocations are made on, with stand-ins for the device: all of them have to
be on the call's stream, between the caller's work there and the kernels."""
import contextlib
import types

import pytest
import torch

import layer_lstm_forward_amd as pkg
from layer_lstm_forward_amd import ops

MAIN, SIDE = 11, 22


class Device(torch.Tensor):
    """A host tensor that says it is on the device and notes where it is copied."""
    is_cuda = property(lambda self: True)

    def contiguous(self, *a, **kw):
        if not self.is_contiguous():
            NOTES.append(("copy", NOW[0]))
        return super().contiguous(*a, **kw)

    def record_stream(self, stream):
        NOTES.append(("given to", stream.cuda_stream))


NOTES, NOW = [], [MAIN]


@pytest.fixture(autouse=True)
def device(monkeypatch):
    NOTES.clear()
    NOW[0] = MAIN

    @contextlib.contextmanager
    def stream(s):
        before, NOW[0] = NOW[0], s.cuda_stream
        yield
        NOW[0] = before

    handle = lambda n: types.SimpleNamespace(cuda_stream=n)  # noqa: E731
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda n, device=None: handle(n))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: handle(NOW[0]))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: NOW[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: None, raising=False)

    def noted(make):
        def f(*a, **kw):
            NOTES.append(("allocation", NOW[0]))
            return make(*a, **kw).as_subclass(Device)
        return f

    for name in ("empty", "empty_like", "tensor"):
        monkeypatch.setattr(torch, name, noted(getattr(torch, name)))
    for name in ("lstm_layer_norm_forward", "lstm_layer_norm_backward", "lstm_linear_attention_forward",
                 "lstm_linear_attention_backward", "lstm_linear_attention_step"):
        monkeypatch.setattr(ops, name, lambda *a: NOTES.append(("kernels", a[-1])) or 0)
    for name in ("lstm_layer_norm_backward_workspace_size", "lstm_linear_attention_workspace_size",
                 "lstm_linear_attention_backward_workspace_size"):
        monkeypatch.setattr(ops, name, lambda *a: 64)


def put(*shape):
    return torch.zeros(*shape).as_subclass(Device)


def check(copies, results):
    """Notes of a call on SIDE from MAIN: `copies` of its arguments and `results` that it allocated."""
    assert NOTES.count(("copy", SIDE)) == copies
    assert NOTES.count(("given to", MAIN)) == results
    assert {n for n in NOTES if n[0] != "given to"} <= {("copy", SIDE), ("allocation", SIDE), ("kernels", SIDE)}
    assert NOW[0] == MAIN
    NOTES.clear()


def test_layer_norm():
    x, res, ds = put(4, 3, 8).transpose(0, 1), put(8, 3, 4).transpose(0, 2).transpose(0, 1), put(4, 3, 8).transpose(0, 1)
    y, mean, rstd, z = pkg.layer_norm(x, residual=res, stream=SIDE)
    check(2, 4)
    pkg.layer_norm_backward(x, x, mean, rstd, dsum=ds, stream=SIDE)
    check(3, 3)
    pkg.layer_norm(x)  # the current stream: no switch, nothing to give
    assert set(NOTES) == {("copy", MAIN), ("allocation", MAIN), ("kernels", MAIN)}


def test_linear_attention():
    q, g, S = put(5, 2, 4, 8), put(4), put(2, 4, 8, 8)
    o, last = pkg.linear_attention(q, q, q, g, lengths=[5, 2], stream=SIDE)
    check(0, 2)
    pkg.linear_attention_backward(q, q, q, g, o, state=S, lengths=[5, 2], stream=SIDE)
    check(0, 4)
    pkg.linear_attention_step(q[0], q[0], q[0], g, S, stream=SIDE)
    check(0, 1)
