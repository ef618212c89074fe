"""Binding of include/lstm_blocks.h: the gated linear recurrence, rotary
positions with the norm of each head, and the gated feed-forward block.

As in ops.py, the ``lstm_*`` functions carry the C ABI's names and take integer
device addresses (0 = NULL); the functions below them take and return torch
tensors and run on the current stream of the tensors' device, or on ``stream``
(an integer ``hipStream_t``), as a call made with that stream as torch's
current one.  There is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import struct

import layer_lstm_forward_amd as _base
from . import ops as _ops
from .ops import (_On, _Struct, _addr, _check, _code, _dense, _lengths, _pack_view, _sequence, _view, _width)

_vp, _i, _sz, _ll, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_float

LSTM_ACT_SILU, LSTM_ACT_GELU, LSTM_ACT_SIGMOID = 0, 1, 2
ACTIVATIONS = {"silu": LSTM_ACT_SILU, "gelu": LSTM_ACT_GELU, "sigmoid": LSTM_ACT_SIGMOID}

torch = None  # imported by the first call of a torch wrapper, as everywhere in this package


def _need_torch():
    global torch
    _ops._need_torch()
    torch = _ops.torch


class lstm_gated_recurrence_shape(ctypes.Structure):
    _fields_ = [("dtype", _i), ("T", _i), ("B", _i), ("width", _i)]


class lstm_rotary_shape(ctypes.Structure):
    _fields_ = [("dtype", _i), ("T", _i), ("B", _i), ("heads", _i), ("kv_heads", _i), ("dim", _i),
                ("rotary_dim", _i), ("interleaved", _i), ("norm", _i), ("eps", _f), ("scale", _f)]


class lstm_positions(ctypes.Structure):
    _fields_ = [("data", _vp), ("time", _ll), ("batch", _ll)]


class lstm_gated_mlp_shape(ctypes.Structure):
    _fields_ = [("dtype", _i), ("activation", _i), ("rows", _i), ("in", _i), ("hidden", _i), ("out", _i)]


_pack_recurrence = struct.Struct("@iiii").pack
_pack_rotary = struct.Struct("@iiiiiiiiiff").pack
_pack_positions = struct.Struct("@Pqq").pack
_pack_mlp = struct.Struct("@iiiiii").pack

_ready = None


def _lib():
    global _ready
    if _ready is not None:
        return _ready
    lib = _base.load_library()
    s, szp = _Struct, ctypes.POINTER(_sz)  # structures travel as their bytes or as ctypes structures
    for name, args in (
            ("lstm_gated_recurrence_workspace_size", [s, szp]),
            ("lstm_gated_recurrence_backward_workspace_size", [s, szp]),
            ("lstm_gated_recurrence_forward", [s, s, s, s, _vp, _vp, s, _vp, _vp, _sz, _vp]),
            ("lstm_gated_recurrence_backward", [s, s, s, s, _vp, _vp, s, s, _vp, s, s, s, _vp, _vp, _sz, _vp]),
            ("lstm_gated_recurrence_step", [s, s, s, s, _vp, _i, _vp, s, _vp]),
            ("lstm_rotary_forward", [s, s, s, _vp, _vp, _vp, s, s, s, _vp]),
            ("lstm_rotary_backward_workspace_size", [s, szp]),
            ("lstm_rotary_backward", [s, s, s, _vp, _vp, _vp, s, s, s, s, s, _vp, _vp, _vp, _sz, _vp]),
            ("lstm_gated_mlp_workspace_size", [s, szp]),
            ("lstm_gated_mlp_reserve_size", [s, szp]),
            ("lstm_gated_mlp_backward_workspace_size", [s, szp]),
            ("lstm_gated_mlp_forward", [s, _vp, _ll, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _sz, _vp]),
            ("lstm_gated_mlp_backward", [s, _vp, _ll, _vp, _vp, _vp, _vp, _sz, _vp, _ll, _vp, _vp, _vp, _vp, _vp, _sz,
                                         _vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = _i, args
    _ready = lib
    return lib


# ------------------------------------------------------------- C-ABI mirror
def _size(name, shape) -> int:
    n = _sz()
    rc = getattr(_lib(), name)(shape, n)
    if rc:
        raise _base.LSTMError(rc, name)
    return n.value


def lstm_gated_recurrence_workspace_size(shape) -> int:
    return _size("lstm_gated_recurrence_workspace_size", shape)


def lstm_gated_recurrence_backward_workspace_size(shape) -> int:
    return _size("lstm_gated_recurrence_backward_workspace_size", shape)


def lstm_gated_recurrence_forward(shape, x, forget, input, lengths, state, y, state_out, workspace, workspace_bytes,
                                  stream) -> int:
    return _lib().lstm_gated_recurrence_forward(shape, x, forget, input, lengths, state, y, state_out, workspace,
                                                workspace_bytes, stream)


def lstm_gated_recurrence_backward(shape, x, forget, input, lengths, state, y, dy, dstate_out, dx, dforget, dinput,
                                   dstate, workspace, workspace_bytes, stream) -> int:
    return _lib().lstm_gated_recurrence_backward(shape, x, forget, input, lengths, state, y, dy, dstate_out, dx,
                                                 dforget, dinput, dstate, workspace, workspace_bytes, stream)


def lstm_gated_recurrence_step(shape, x, forget, input, slots, n_slots, pool, y, stream) -> int:
    return _lib().lstm_gated_recurrence_step(shape, x, forget, input, slots, n_slots, pool, y, stream)


def lstm_rotary_forward(shape, q, k, q_weight, k_weight, frequencies, positions, q_out, k_out, stream) -> int:
    return _lib().lstm_rotary_forward(shape, q, k, q_weight, k_weight, frequencies, positions, q_out, k_out, stream)


def lstm_rotary_backward_workspace_size(shape) -> int:
    return _size("lstm_rotary_backward_workspace_size", shape)


def lstm_rotary_backward(shape, q, k, q_weight, k_weight, frequencies, positions, dq_out, dk_out, dq, dk, dq_weight,
                         dk_weight, workspace, workspace_bytes, stream) -> int:
    return _lib().lstm_rotary_backward(shape, q, k, q_weight, k_weight, frequencies, positions, dq_out, dk_out, dq,
                                       dk, dq_weight, dk_weight, workspace, workspace_bytes, stream)


def lstm_gated_mlp_workspace_size(shape) -> int:
    return _size("lstm_gated_mlp_workspace_size", shape)


def lstm_gated_mlp_reserve_size(shape) -> int:
    return _size("lstm_gated_mlp_reserve_size", shape)


def lstm_gated_mlp_backward_workspace_size(shape) -> int:
    return _size("lstm_gated_mlp_backward_workspace_size", shape)


def lstm_gated_mlp_forward(shape, x, x_stride, w_gate, w_up, w_down, y, reserve, reserve_bytes, workspace,
                           workspace_bytes, stream) -> int:
    return _lib().lstm_gated_mlp_forward(shape, x, x_stride, w_gate, w_up, w_down, y, reserve, reserve_bytes,
                                         workspace, workspace_bytes, stream)


def lstm_gated_mlp_backward(shape, x, x_stride, w_gate, w_up, w_down, reserve, reserve_bytes, dy, dy_stride, dx,
                            dw_gate, dw_up, dw_down, workspace, workspace_bytes, stream) -> int:
    return _lib().lstm_gated_mlp_backward(shape, x, x_stride, w_gate, w_up, w_down, reserve, reserve_bytes, dy,
                                          dy_stride, dx, dw_gate, dw_up, dw_down, workspace, workspace_bytes, stream)


def _output(t, like, what, shape):
    """A tensor to write into: as _sequence, and no two of its elements in one place."""
    _sequence(t, like, what, shape)
    if any(n > 1 and s == 0 for n, s in zip(shape, t.stride())):
        raise ValueError(f"{what} must not be an expanded tensor: it is written")


# ---------------------------------------------------------- gated recurrence
def _channels(t, batch_first):
    """The view of a [T, B, width] tensor."""
    s = t.stride()
    return _pack_view(t.data_ptr(), s[1], s[0], 0) if batch_first else _pack_view(t.data_ptr(), s[0], s[1], 0)


def _recurrence_args(x, forget, input_gate, state, lead_axes, what):
    code = _code(x, "x")
    size = x.shape
    if len(size) != lead_axes + 1:
        raise ValueError(f"x must be {what}")
    _sequence(x, x, "x", size)
    _sequence(forget, x, "forget", size)
    if input_gate is not None:
        _sequence(input_gate, x, "input_gate", size)
    return code


def gated_recurrence(x, forget, input_gate=None, state=None, lengths=None, batch_first=False, out=None, stream=None):
    """h_t = a_t h_{t-1} + w_t x_t for every channel over sequences (lstm_gated_recurrence_forward), with the logistic
    function s, a_t = s(forget_t) and w_t = s(input_gate_t), or 1 - a_t without an input gate.

    x, forget, input_gate [T, B, width] ([B, T, width] with batch_first), any strides with a dense last axis (slices
    of one wide projection need no copy).  state: None or [B, width] float32, from an earlier call.
    lengths: None, B host ints in 0..T, or an int32 device tensor; tokens past a row's length are not read.
    out: None or (y, state_out) to write into; y must not share memory with an input, state_out may be `state`.
    Returns (y, state_out); y holds every h_t."""
    if torch is None:
        _need_torch()
    code = _recurrence_args(x, forget, input_gate, state, 2, "[T, B, width] ([B, T, width] with batch_first)")
    T, B = (x.shape[1], x.shape[0]) if batch_first else x.shape[:2]
    width = x.shape[2]
    if state is not None:
        _dense(state, x, "state", (B, width), torch.float32)
    shape = _pack_recurrence(code, T, B, width)
    with _On(x.device, stream) as on:
        lens = _lengths(lengths, T, B, x.device)
        if out is None:
            y = x.new_empty(x.shape)
            last = torch.empty(B, width, dtype=torch.float32, device=x.device)
            if on.other is not None:
                on.give(y, last)
        else:
            y, last = out
            _output(y, x, "y", x.shape)
            if last is not None:
                _dense(last, x, "state_out", (B, width), torch.float32)
        nbytes = lstm_gated_recurrence_workspace_size(shape)
        ws = on.scratch(nbytes)
        _check(lstm_gated_recurrence_forward(
            shape, _channels(x, batch_first), _channels(forget, batch_first),
            None if input_gate is None else _channels(input_gate, batch_first), _addr(lens), _addr(state),
            _channels(y, batch_first), _addr(last), _addr(ws), nbytes, on.handle), "lstm_gated_recurrence_forward")
    return y, last


def gated_recurrence_backward(x, forget, y, dy, input_gate=None, state=None, dstate=None, lengths=None,
                              batch_first=False, out=None, stream=None):
    """Gradients (dx, dforget, dinput_gate, dstate) of gated_recurrence() called with the same arguments.

    y: as that call returned it; dy: its gradient; dstate: gradient of the returned state, or None.  out: None or (dx,
    dforget, dinput_gate) to write into, which must not share memory with an input.  dinput_gate and the last result,
    the gradient of `state`, are None where there was none."""
    if torch is None:
        _need_torch()
    code = _recurrence_args(x, forget, input_gate, state, 2, "[T, B, width] ([B, T, width] with batch_first)")
    T, B = (x.shape[1], x.shape[0]) if batch_first else x.shape[:2]
    width = x.shape[2]
    _sequence(y, x, "y", x.shape)
    _sequence(dy, x, "dy", x.shape)
    for t, what in ((state, "state"), (dstate, "dstate")):
        if t is not None:
            _dense(t, x, what, (B, width), torch.float32)
    shape = _pack_recurrence(code, T, B, width)
    with _On(x.device, stream) as on:
        lens = _lengths(lengths, T, B, x.device)
        if out is None:
            dx, df = x.new_empty(x.shape), x.new_empty(x.shape)
            di = None if input_gate is None else x.new_empty(x.shape)
            if on.other is not None:
                on.give(dx, df, di)
        else:
            dx, df, di = out
            if (di is None) != (input_gate is None):
                raise ValueError("dinput_gate must be given exactly where input_gate is")
            for t, what in ((dx, "dx"), (df, "dforget"), (di, "dinput_gate")):
                if t is not None:
                    _output(t, x, what, x.shape)
        dfirst = None if state is None else torch.empty_like(state)
        if on.other is not None:
            on.give(dfirst)
        nbytes = lstm_gated_recurrence_backward_workspace_size(shape)
        ws = on.scratch(nbytes)
        view = lambda t: None if t is None else _channels(t, batch_first)  # noqa: E731
        _check(lstm_gated_recurrence_backward(
            shape, view(x), view(forget), view(input_gate), _addr(lens), _addr(state), view(y), view(dy),
            _addr(dstate), view(dx), view(df), view(di), _addr(dfirst), _addr(ws), nbytes, on.handle),
            "lstm_gated_recurrence_backward")
    return dx, df, di, dfirst


def gated_recurrence_step(x, forget, state, input_gate=None, slots=None, out=None, stream=None):
    """One token for each of B requests (lstm_gated_recurrence_step); returns y [B, width].

    x, forget, input_gate [B, width].  state [n, width] float32 is updated in place.  slots: None (row b is state[b])
    or B int32 values on the device: row b is state[slots[b]], and a value outside 0..n-1 marks an idle row, whose y
    is 0; no two rows may name the same slot."""
    if torch is None:
        _need_torch()
    code = _recurrence_args(x, forget, input_gate, state, 1, "[B, width]")
    B, width = x.shape
    if state.dim() != 2:
        raise ValueError("state must be [n, width]")
    _dense(state, x, "state", (state.shape[0], width), torch.float32)
    if slots is not None:
        _dense(slots, x, "slots", (B,), torch.int32)
    with _On(x.device, stream) as on:
        if out is None:
            out = x.new_empty(x.shape)
            if on.other is not None:
                on.give(out)
        else:
            _output(out, x, "y", x.shape)
        view = lambda t: None if t is None else _pack_view(t.data_ptr(), 0, t.stride(0), 0)  # noqa: E731
        _check(lstm_gated_recurrence_step(_pack_recurrence(code, 1, B, width), view(x), view(forget),
                                          view(input_gate), _addr(slots), state.shape[0], state.data_ptr(), view(out),
                                          on.handle), "lstm_gated_recurrence_step")
    return out


# -------------------------------------------------------------------- rotary
def rotary_frequencies(rotary_dim, base=10000.0, factor=1.0, original_length=None, low=1.0, high=4.0, device="cuda"):
    """The rotary_dim / 2 frequencies base ** (-2 j / rotary_dim), radians a position, as rotary() takes them: float64.

    factor: how many times longer than in training texts become.  Without original_length every frequency is divided by
    it (positions are interpolated).  With it, a frequency that makes at least `high` turns in a text of original_length
    stays as it is, one that makes at most `low` is divided, and between them the two are mixed in proportion."""
    if torch is None:
        _need_torch()
    if rotary_dim < 0 or rotary_dim % 2 or not base > 0 or not factor > 0:
        raise ValueError("rotary_dim must be even, base and factor positive")
    if original_length is not None and not (original_length > 0 and high > low):
        raise ValueError("original_length must be positive and high above low")
    out = []
    for j in range(rotary_dim // 2):
        f = float(base) ** (-2.0 * j / rotary_dim)
        keep = 0.0
        if original_length is not None:
            keep = min(1.0, max(0.0, (original_length * f / (2 * math.pi) - low) / (high - low)))
        out.append(f * (keep + (1.0 - keep) / factor))
    return torch.tensor(out, dtype=torch.float64, device=device)


def _float32(value, what):
    """A number as the ABI's float holds it, refused where it would become 0 or infinite there."""
    value = float(value)
    held = ctypes.c_float(value).value
    if (held == 0.0 and value != 0.0) or (math.isinf(held) and not math.isinf(value)):
        raise ValueError(f"{what} is outside the float32 range")
    return value


class _Rotary:
    """The checked arguments of a call, as the ABI takes them."""

    __slots__ = ("lead", "shape", "positions", "view")

    def __init__(self, q, k, frequencies, positions, q_weight, k_weight, norm, eps, interleaved, scale, batch_first):
        code = _code(q, "q")
        size = q.shape
        if len(size) not in (3, 4):
            raise ValueError("q must be [T, B, heads, dim] ([B, T, heads, dim] with batch_first), or [B, heads, dim]")
        self.lead = lead = size[:-2]
        H, D = size[-2:]
        _sequence(q, q, "q", size)
        G = 0
        if k is not None:
            if k.dim() != len(size):
                raise ValueError("q and k must have as many axes")
            G = k.shape[-2]
            _sequence(k, q, "k", lead + (G, D))
        if len(lead) == 1:
            T, B = 1, lead[0]
            self.view = lambda t: None if t is None else _pack_view(t.data_ptr(), 0, *t.stride()[:2])
        else:
            T, B = (lead[1], lead[0]) if batch_first else lead
            self.view = lambda t: None if t is None else _view(t, batch_first)
        if frequencies.dim() != 1:
            raise ValueError("frequencies must be one axis of float64 values")
        _dense(frequencies, q, "frequencies", frequencies.shape, torch.float64)
        if q_weight is not None or k_weight is not None:
            if not norm:
                raise ValueError("q_weight and k_weight need norm=True")
            for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
                if w is not None:
                    _dense(w, q, what, (D,))
        self.positions = None
        if positions is not None:
            if positions.dtype != torch.int32 or positions.device != q.device or positions.shape != lead:
                raise ValueError(f"positions must be an int32 tensor of shape {list(lead)} on {q.device}")
            s = positions.stride()
            t, b = (0, s[0]) if len(lead) == 1 else (s[1], s[0]) if batch_first else s
            self.positions = _pack_positions(positions.data_ptr(), t, b)
        self.shape = _pack_rotary(code, T, B, H, G, D, 2 * frequencies.shape[0], int(bool(interleaved)),
                                  int(bool(norm)), _float32(eps, "eps"), _float32(scale, "scale"))


def rotary(q, k, frequencies, positions=None, q_weight=None, k_weight=None, norm=False, eps=1e-6, interleaved=False,
           scale=1.0, batch_first=False, out=None, stream=None):
    """Queries and keys of a layer turned by their tokens' positions, after the norm of each head with norm=True
    (lstm_rotary_forward); returns (q, k), in new tensors.

    q [T, B, heads, dim] ([B, T, heads, dim] with batch_first, [B, heads, dim] for single tokens), k with heads of its
    own number, or None; any strides with a dense last axis.  frequencies: as rotary_frequencies makes them; the first
    2 * len(frequencies) values of each head are turned, value j with value j + len(frequencies), or neighbours with
    interleaved=True.  positions: int32, of q's leading axes, any strides, or None (token t of a row stands at t).
    norm=True: x / sqrt(mean(x^2) + eps) * weight first, weights [dim] or None (ones).
    scale: the turned values are multiplied by it.  out: None or (q, k) to write into, each of which may be its input
    itself and must not share memory with anything else."""
    if torch is None:
        _need_torch()
    a = _Rotary(q, k, frequencies, positions, q_weight, k_weight, norm, eps, interleaved, scale, batch_first)
    with _On(q.device, stream) as on:
        if out is None:
            qo = q.new_empty(q.shape)
            ko = None if k is None else k.new_empty(k.shape)
            if on.other is not None:
                on.give(qo, ko)
        else:
            qo, ko = out
            _output(qo, q, "q of out", q.shape)
            if k is not None:
                _output(ko, q, "k of out", k.shape)
        _check(lstm_rotary_forward(a.shape, a.view(q), a.view(k), _addr(q_weight), _addr(k_weight),
                                   frequencies.data_ptr(), a.positions, a.view(qo), a.view(ko), on.handle),
               "lstm_rotary_forward")
    return qo, ko


def rotary_backward(q, k, frequencies, dq_out, dk_out, positions=None, q_weight=None, k_weight=None, norm=False,
                    eps=1e-6, interleaved=False, scale=1.0, batch_first=False, out=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of rotary() called with the same arguments.

    dq_out, dk_out: gradients of its results.  out: None or (dq, dk) to write into, which may be dq_out and dk_out
    themselves and must not share memory with anything else.  The weights' gradients are None without a norm; with
    norm=True they are given without weights too (the gradients of ones)."""
    if torch is None:
        _need_torch()
    a = _Rotary(q, k, frequencies, positions, q_weight, k_weight, norm, eps, interleaved, scale, batch_first)
    _sequence(dq_out, q, "dq_out", q.shape)
    if k is not None:
        _sequence(dk_out, q, "dk_out", k.shape)
    with _On(q.device, stream) as on:
        if out is None:
            dq = q.new_empty(q.shape)
            dk = None if k is None else k.new_empty(k.shape)
            if on.other is not None:
                on.give(dq, dk)
        else:
            dq, dk = out
            _output(dq, q, "dq", q.shape)
            if k is not None:
                _output(dk, q, "dk", k.shape)
        dwq = dwk = None
        if norm:
            dwq = q.new_empty(q.shape[-1])
            if k is not None:  # (keys of no heads are not read, and sum up to nothing)
                dwk = q.new_empty(q.shape[-1]) if k.shape[-2] else q.new_zeros(q.shape[-1])
            if on.other is not None:
                on.give(dwq, dwk)
        nbytes = lstm_rotary_backward_workspace_size(a.shape)
        ws = on.scratch(nbytes)
        _check(lstm_rotary_backward(a.shape, a.view(q), a.view(k), _addr(q_weight), _addr(k_weight),
                                    frequencies.data_ptr(), a.positions, a.view(dq_out),
                                    None if k is None else a.view(dk_out), a.view(dq),
                                    None if k is None else a.view(dk), _addr(dwq), _addr(dwk), _addr(ws), nbytes,
                                    on.handle), "lstm_rotary_backward")
    return dq, dk, dwq, dwk


# ----------------------------------------------------------------- gated MLP
def _tokens(t, what):
    """A tensor whose leading axes are evenly spaced rows (copied if they are not), the spacing, and their number."""
    width = _width(t, what)
    if t.numel() == 0:
        return t, width, 0
    if t.is_contiguous():
        return t, width, t.numel() // width
    if t.dim() != 2 or (width > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < width):
        return t.contiguous(), width, t.numel() // width
    return t, max(t.stride(0), width), t.shape[0]


class _Mlp:
    """The checked weights of a call and its shape."""

    __slots__ = ("x", "stride", "rows", "shape", "weights", "out")

    def __init__(self, x, w_gate, w_up, w_down, activation):
        code = _code(x, "x")
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}")
        width = _width(x, "x")
        if w_gate.dim() != 2 or w_down.dim() != 2:
            raise ValueError("w_gate and w_up must be [hidden, in], w_down [out, hidden]")
        hidden, self.out = w_gate.shape[0], w_down.shape[0]
        _dense(w_gate, x, "w_gate", (hidden, width))
        _dense(w_up, x, "w_up", (hidden, width))
        _dense(w_down, x, "w_down", (self.out, hidden))
        # the kernels read weights in pieces of 16 bytes
        self.weights = [w if w.data_ptr() % 16 == 0 else w.clone() for w in (w_gate, w_up, w_down)]
        self.x, self.stride, self.rows = _tokens(x, "x")
        self.shape = _pack_mlp(code, ACTIVATIONS[activation], self.rows, width, hidden, self.out)


def _mlp_forward(x, w_gate, w_up, w_down, activation, keep, stream):
    if torch is None:
        _need_torch()
    _code(x, "x")
    with _On(x.device, stream) as on:
        a = _Mlp(x, w_gate, w_up, w_down, activation)
        y = x.new_empty(x.shape[:-1] + (a.out,))
        held = lstm_gated_mlp_reserve_size(a.shape) if keep else 0
        reserve = torch.empty(held, dtype=torch.uint8, device=x.device) if keep else None
        nbytes = lstm_gated_mlp_workspace_size(a.shape)
        ws = on.scratch(nbytes)
        if on.other is not None:
            on.give(y, reserve)
        _check(lstm_gated_mlp_forward(a.shape, a.x.data_ptr(), a.stride, *(w.data_ptr() for w in a.weights),
                                      y.data_ptr(), _addr(reserve), held, _addr(ws), nbytes, on.handle),
               "lstm_gated_mlp_forward")
    return y, reserve


def gated_mlp(x, w_gate, w_up, w_down, activation="silu", stream=None):
    """The gated feed-forward block y = (act(x w_gate^T) * (x w_up^T)) w_down^T (lstm_gated_mlp_forward).

    x [..., in], w_gate and w_up [hidden, in], w_down [out, hidden]; activation "silu", "gelu" (its tanh form) or
    "sigmoid".  Returns y [..., out].  Weights whose address is no multiple of 16 bytes are copied in every call, and so
    is an x whose leading axes are not evenly spaced rows.  The products are summed in 32 bits; bfloat16: the hidden
    values are rounded once as an operand of the last product; float32: operands are split so that products keep 24
    bits."""
    return _mlp_forward(x, w_gate, w_up, w_down, activation, False, stream)[0]


def gated_mlp_train(x, w_gate, w_up, w_down, activation="silu", stream=None):
    """gated_mlp() that keeps what gated_mlp_backward() reads; returns (y, reserve)."""
    return _mlp_forward(x, w_gate, w_up, w_down, activation, True, stream)


def gated_mlp_backward(dy, x, w_gate, w_up, w_down, reserve, activation="silu", stream=None):
    """Gradients (dx, dw_gate, dw_up, dw_down) of gated_mlp_train() called with the same arguments, from the gradient dy
    of its y and its reserve (not changed)."""
    if torch is None:
        _need_torch()
    _code(x, "x")
    with _On(x.device, stream) as on:
        a = _Mlp(x, w_gate, w_up, w_down, activation)
        _ops._same(dy, x, "dy", x.shape[:-1] + (a.out,))
        d, ds, _ = _tokens(dy, "dy")
        held = lstm_gated_mlp_reserve_size(a.shape)
        if reserve.dtype != torch.uint8 or reserve.device != x.device or reserve.numel() != held \
                or not reserve.is_contiguous():
            raise ValueError("reserve must be as gated_mlp_train returned it for this x")
        dx = x.new_empty(x.shape)
        dws = [w.new_empty(w.shape) for w in (w_gate, w_up, w_down)]
        nbytes = lstm_gated_mlp_backward_workspace_size(a.shape)
        ws = on.scratch(nbytes)
        if on.other is not None:
            on.give(dx, *dws)
        _check(lstm_gated_mlp_backward(a.shape, a.x.data_ptr(), a.stride, *(w.data_ptr() for w in a.weights),
                                       reserve.data_ptr(), held, d.data_ptr(), ds, dx.data_ptr(),
                                       *(w.data_ptr() for w in dws), _addr(ws), nbytes, on.handle),
               "lstm_gated_mlp_backward")
    return dx, *dws
