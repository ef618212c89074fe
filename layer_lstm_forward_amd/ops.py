"""Binding of include/lstm_ops.h: linear attention with a decay for each head,
layer norm, and the AdamW step over many tensors.

The ``lstm_*`` functions carry the C ABI's names and take integer device
addresses (0 = NULL).  The functions below them take and return torch tensors
and run on the current stream of the tensors' device, or on ``stream`` (an
integer ``hipStream_t``): a call with ``stream`` is one made with that stream
as torch's current one, copies and allocations included.  The arguments have to
be ready on that stream and are the caller's to keep until it has passed the
call.  As everywhere in this package torch provides device memory and streams
only, and there is no fallback.
"""
from __future__ import annotations

import ctypes
import struct

import layer_lstm_forward_amd as _base

_vp, _i, _sz, _ll, _f, _d = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_float,
                             ctypes.c_double)

LSTM_ADAMW_BLOCK = 256

torch = None  # imported by the first call of a torch wrapper, as everywhere in this package


def _need_torch():
    global torch
    import torch as t
    torch = t


class lstm_view(ctypes.Structure):
    _fields_ = [("data", _vp), ("time", _ll), ("batch", _ll), ("head", _ll)]


class lstm_linear_attention_shape(ctypes.Structure):
    _fields_ = [("dtype", _i), ("T", _i), ("B", _i), ("heads", _i), ("kv_heads", _i), ("key_dim", _i),
                ("value_dim", _i), ("scale", _f)]


class lstm_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", _vp), ("grad", _vp), ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp),
                ("master", _vp), ("n", _ll), ("lr", _f), ("weight_decay", _f)]


class _Struct:
    """Argument type of a structure passed by address: its bytes, a ctypes structure, or None."""

    @classmethod
    def from_param(cls, x):
        if x is None or isinstance(x, bytes):
            return ctypes.c_char_p(x)
        return ctypes.byref(x)


# a structure's bytes cost a third of the ctypes object to make
_pack_view = struct.Struct("@Pqqq").pack
_pack_shape = struct.Struct("@iiiiiiif").pack
_pack_tensor = struct.Struct("@PPPPPPPqff").pack

_ready = None


def _lib():
    global _ready
    if _ready is not None:
        return _ready
    lib = _base.load_library()
    # structures travel as their bytes (see _pack_view) or as ctypes structures
    shape, view, szp = _Struct, _Struct, ctypes.POINTER(_sz)
    for name, args in (
            ("lstm_linear_attention_workspace_size", [shape, szp]),
            ("lstm_linear_attention_backward_workspace_size", [shape, szp]),
            ("lstm_linear_attention_forward", [shape, view, view, view, _vp, _vp, _vp, view, _vp, _vp, _sz, _vp]),
            ("lstm_linear_attention_backward", [shape, view, view, view, _vp, _vp, _vp, view, _vp, view, view, view,
                                                _vp, _vp, _sz, _vp]),
            ("lstm_linear_attention_step", [shape, view, view, view, _vp, _vp, _i, _vp, view, _vp]),
            ("lstm_layer_norm_forward", [_i, _vp, _ll, _vp, _ll, _vp, _vp, _ll, _i, _f, _vp, _vp, _vp, _vp, _vp]),
            ("lstm_layer_norm_backward_workspace_size", [_ll, _i, szp]),
            ("lstm_layer_norm_backward", [_i, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _vp, _ll, _i, _vp, _vp, _vp, _vp,
                                          _sz, _vp]),
            ("lstm_adamw_step", [_i, _i, _Struct, _i, _d, _d, _d, _ll, _vp,
                                 ctypes.c_uint, _vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = _i, args
    _ready = lib
    return lib


# ------------------------------------------------------------- C-ABI mirror
def lstm_linear_attention_workspace_size(shape) -> int:
    n = _sz()
    rc = _lib().lstm_linear_attention_workspace_size(shape, n)
    if rc:
        raise _base.LSTMError(rc, "lstm_linear_attention_workspace_size")
    return n.value


def lstm_linear_attention_backward_workspace_size(shape) -> int:
    n = _sz()
    rc = _lib().lstm_linear_attention_backward_workspace_size(shape, n)
    if rc:
        raise _base.LSTMError(rc, "lstm_linear_attention_backward_workspace_size")
    return n.value


def lstm_linear_attention_forward(shape, q, k, v, log_decay, lengths, state, o, state_out, workspace,
                                  workspace_bytes, stream) -> int:
    return _lib().lstm_linear_attention_forward(shape, q, k, v, log_decay, lengths, state, o, state_out, workspace,
                                                workspace_bytes, stream)


def lstm_linear_attention_backward(shape, q, k, v, log_decay, lengths, state, do, dstate_out, dq, dk, dv, dstate,
                                   workspace, workspace_bytes, stream) -> int:
    return _lib().lstm_linear_attention_backward(shape, q, k, v, log_decay, lengths, state, do, dstate_out, dq, dk,
                                                 dv, dstate, workspace, workspace_bytes, stream)


def lstm_linear_attention_step(shape, q, k, v, log_decay, slots, n_slots, pool, o, stream) -> int:
    return _lib().lstm_linear_attention_step(shape, q, k, v, log_decay, slots, n_slots, pool, o, stream)


def lstm_layer_norm_forward(dtype, x, x_stride, residual, residual_stride, weight, bias, rows, width, eps, y, sum,
                            mean, rstd, stream) -> int:
    return _lib().lstm_layer_norm_forward(dtype, x, x_stride, residual, residual_stride, weight, bias, rows, width,
                                          eps, y, sum, mean, rstd, stream)


def lstm_layer_norm_backward_workspace_size(rows, width) -> int:
    n = _sz()
    rc = _lib().lstm_layer_norm_backward_workspace_size(rows, width, n)
    if rc:
        raise _base.LSTMError(rc, "lstm_layer_norm_backward_workspace_size")
    return n.value


def lstm_layer_norm_backward(dtype, dy, dy_stride, z, z_stride, mean, rstd, weight, dsum, rows, width, dx, dweight,
                             dbias, workspace, workspace_bytes, stream) -> int:
    return _lib().lstm_layer_norm_backward(dtype, dy, dy_stride, z, z_stride, mean, rstd, weight, dsum, rows, width,
                                           dx, dweight, dbias, workspace, workspace_bytes, stream)


def lstm_adamw_step(dtype, state_bits, tensors, count, beta1, beta2, eps, step, grad_scale, seed, stream) -> int:
    """tensors: a ctypes array of lstm_adamw_tensor, or its bytes."""
    return _lib().lstm_adamw_step(dtype, state_bits, tensors, count, beta1, beta2, eps, step, grad_scale, seed,
                                  stream)


# ------------------------------------------------------------ torch wrappers
def _check(rc, where):
    if rc:
        raise _base.LSTMError(rc, where)


def _code(t, what):
    """The ABI's dtype code of a device tensor."""
    if t.is_cuda:
        if t.dtype == torch.bfloat16:
            return _base.LSTM_BF16
        if t.dtype == torch.float32:
            return _base.LSTM_F32
    raise ValueError(f"{what} must be a float32 or bfloat16 device tensor")


def _same(t, like, what, shape=None):
    if t.dtype != like.dtype or t.device != like.device or (shape is not None and t.shape != shape):
        raise ValueError(f"{what} must be of {like.dtype} on {like.device}"
                         + (f" and of shape {list(shape)}" if shape is not None else ""))


def _dense(t, like, what, shape, dtype=None):
    if t.device != like.device or t.dtype != (dtype or like.dtype) or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype or like.dtype} tensor of shape {list(shape)} "
                         f"on {like.device}")


def _addr(t):
    return None if t is None else t.data_ptr()


class _On:
    """The stream of a call.  Where it is not torch's current one it becomes that for the call (a `with` block), so
    that copies and memory of the call come in the kernels' order: a block that torch hands out for the current stream
    may still be in use there, and a copy made there may run before its source is written or after it is read."""

    __slots__ = ("device", "handle", "other", "_current", "_guard")

    def __init__(self, device, stream):
        self.device = device
        self.handle = torch._C._cuda_getCurrentRawStream(device.index)
        self.other = None
        if stream is not None and int(stream) != self.handle:
            self.handle = int(stream)
            self.other = torch.cuda.ExternalStream(self.handle, device)
            self._current = torch.cuda.current_stream(device)

    def __enter__(self):
        self._guard = None
        if self.other is not None:
            self._guard = torch.cuda.stream(self.other)
        elif torch._C._cuda_getDevice() != self.device.index:
            self._guard = torch.cuda.device(self.device)
        if self._guard is not None:
            self._guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)

    def give(self, *results):
        """For results of a call on another stream: the caller's work on the current one may read them, too, so their
        memory is not handed out again before that stream has passed what it had queued when they were dropped."""
        for t in results:
            if t is not None:
                t.record_stream(self._current)

    def scratch(self, nbytes):
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None


def _view(t, batch_first):
    s = t.stride()
    return _pack_view(t.data_ptr(), s[1], s[0], s[2]) if batch_first else _pack_view(t.data_ptr(), *s[:3])


def _sequence(t, like, what, shape):
    """A [.., heads, dim] tensor whose last axis is dense."""
    if t.shape != shape or t.dtype != like.dtype or t.device != like.device or (shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{what} must be a {like.dtype} tensor of shape {list(shape)} on {like.device}, "
                         "its last axis dense")


class _Shape:
    """The sizes of a call, checked against its tensors, and as the ABI takes them."""

    __slots__ = ("heads", "key_dim", "value_dim", "B", "packed")

    def __init__(self, q, k, v, log_decay, scale, lead, T, B):
        code = _code(q, "q")
        H, Dk = q.shape[-2:]
        if k.dim() != q.dim() or v.dim() != q.dim():
            raise ValueError("q, k and v must have as many axes")
        G, Dv = v.shape[-2:]
        _sequence(q, q, "q", lead + (H, Dk))
        _sequence(k, q, "k", lead + (G, Dk))
        _sequence(v, q, "v", lead + (G, Dv))
        if log_decay.dtype != torch.float32 or log_decay.shape != (H,) or log_decay.device != q.device \
                or not log_decay.is_contiguous():
            raise ValueError(f"log_decay must be {H} contiguous float32 values on {q.device}")
        self.heads, self.key_dim, self.value_dim, self.B = H, Dk, Dv, B
        self.packed = _pack_shape(code, T, B, H, G, Dk, Dv, (Dk or 1) ** -0.5 if scale is None else scale)


def _lengths(lengths, T, B, device):
    """None, B host ints (each checked), or an int32 device tensor (each clamped to 0..T on the device)."""
    if lengths is None:
        return None
    if isinstance(lengths, torch.Tensor) and lengths.is_cuda:
        if lengths.dtype != torch.int32 or tuple(lengths.shape) != (B,) or lengths.device != device \
                or not lengths.is_contiguous():
            raise ValueError(f"lengths must be {B} int32 values on {device}, or host ints")
        return lengths
    values = [int(n) for n in lengths]
    if len(values) != B or any(n < 0 or n > T for n in values):
        raise ValueError(f"lengths must be {B} values in 0..{T}")
    return torch.tensor(values, dtype=torch.int32, device=device)


def _state_check(state, q, shape, what):
    if state is not None:
        _dense(state, q, what, (shape.B, shape.heads, shape.key_dim, shape.value_dim), torch.float32)


def linear_attention(q, k, v, log_decay, scale=None, state=None, lengths=None, batch_first=False, out=None,
                     stream=None):
    """S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale q_t S_t over sequences (lstm_linear_attention_forward).

    q [T, B, heads, key_dim] ([B, T, heads, key_dim] with batch_first), k and v with kv_heads heads, which may be
    fewer: each is then shared by heads / kv_heads query heads.  Any strides with a dense last axis (slices of one
    wide projection need no copy).  log_decay [heads] float32.  scale: key_dim ** -0.5 unless given.
    state: None or [B, heads, key_dim, value_dim] float32, from an earlier call.
    lengths: None, B host ints in 0..T, or an int32 device tensor; tokens past a row's length are not read.
    out: None or (o, state_out) to write into; state_out may be `state`.
    bfloat16: the state, where tokens read it, and the products of a chunk's queries and keys are rounded as operands
    (linear_attention_step rounds its result alone).
    Returns (o, state_out)."""
    if torch is None:
        _need_torch()
    if q.dim() != 4:
        raise ValueError("q must be [T, B, heads, key_dim] ([B, T, heads, key_dim] with batch_first)")
    lead = tuple(q.shape[:2])
    T, B = (lead[1], lead[0]) if batch_first else lead
    shape = _Shape(q, k, v, log_decay, scale, lead, T, B)
    _state_check(state, q, shape, "state")
    with _On(q.device, stream) as on:
        lens = _lengths(lengths, T, B, q.device)
        if out is None:
            o = torch.empty(*lead, shape.heads, shape.value_dim, dtype=q.dtype, device=q.device)
            last = torch.empty(B, shape.heads, shape.key_dim, shape.value_dim, dtype=torch.float32, device=q.device)
            if on.other is not None:
                on.give(o, last)
        else:
            o, last = out
            _sequence(o, q, "o", lead + (shape.heads, shape.value_dim))
            _state_check(last, q, shape, "state_out")
        nbytes = lstm_linear_attention_workspace_size(shape.packed)
        ws = on.scratch(nbytes)
        _check(lstm_linear_attention_forward(shape.packed, _view(q, batch_first), _view(k, batch_first),
                                             _view(v, batch_first), log_decay.data_ptr(), _addr(lens), _addr(state),
                                             _view(o, batch_first), _addr(last), _addr(ws), nbytes, on.handle),
               "lstm_linear_attention_forward")
    return o, last


def linear_attention_backward(q, k, v, log_decay, do, scale=None, state=None, dstate=None, lengths=None,
                              batch_first=False, out=None, stream=None):
    """Gradients (dq, dk, dv, dstate) of linear_attention() called with the same arguments.

    do: gradient of o; dstate: gradient of the returned state, or None.  out: None or (dq, dk, dv) to write into.
    The last result is the gradient of `state`, or None where there was none."""
    if torch is None:
        _need_torch()
    if q.dim() != 4:
        raise ValueError("q must be [T, B, heads, key_dim] ([B, T, heads, key_dim] with batch_first)")
    lead = tuple(q.shape[:2])
    T, B = (lead[1], lead[0]) if batch_first else lead
    shape = _Shape(q, k, v, log_decay, scale, lead, T, B)
    _sequence(do, q, "do", lead + (shape.heads, shape.value_dim))
    _state_check(state, q, shape, "state")
    _state_check(dstate, q, shape, "dstate")
    with _On(q.device, stream) as on:
        lens = _lengths(lengths, T, B, q.device)
        if out is None:
            dq, dk, dv = (torch.empty(t.shape, dtype=q.dtype, device=q.device) for t in (q, k, v))
            if on.other is not None:
                on.give(dq, dk, dv)
        else:
            dq, dk, dv = out
            for t, like, what in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
                _sequence(t, q, what, like.shape)
        dfirst = None if state is None else torch.empty_like(state)
        if on.other is not None:
            on.give(dfirst)
        nbytes = lstm_linear_attention_backward_workspace_size(shape.packed)
        ws = on.scratch(nbytes)
        _check(lstm_linear_attention_backward(
            shape.packed, _view(q, batch_first), _view(k, batch_first), _view(v, batch_first), log_decay.data_ptr(),
            _addr(lens), _addr(state), _view(do, batch_first), _addr(dstate), _view(dq, batch_first),
            _view(dk, batch_first), _view(dv, batch_first), _addr(dfirst), _addr(ws), nbytes, on.handle),
            "lstm_linear_attention_backward")
    return dq, dk, dv, dfirst


def linear_attention_step(q, k, v, log_decay, state, scale=None, slots=None, out=None, stream=None):
    """One token for each of B requests (lstm_linear_attention_step); returns o [B, heads, value_dim].

    q [B, heads, key_dim], k and v with kv_heads heads.  state [n, heads, key_dim, value_dim] float32 is updated in
    place.  slots: None (row b is state[b]) or B int32 values on the device: row b is state[slots[b]], and a value
    outside 0..n-1 marks an idle row, whose o is 0; no two rows may name the same slot."""
    if torch is None:
        _need_torch()
    if q.dim() != 3:
        raise ValueError("q must be [B, heads, key_dim]")
    B = q.shape[0]
    shape = _Shape(q, k, v, log_decay, scale, (B,), 1, B)
    if state.dim() != 4:
        raise ValueError("state must be [n, heads, key_dim, value_dim]")
    _dense(state, q, "state", (state.shape[0], shape.heads, shape.key_dim, shape.value_dim), torch.float32)
    if slots is not None:
        _dense(slots, q, "slots", (B,), torch.int32)
    with _On(q.device, stream) as on:
        if out is None:
            out = torch.empty(B, shape.heads, shape.value_dim, dtype=q.dtype, device=q.device)
            if on.other is not None:
                on.give(out)
        else:
            _sequence(out, q, "o", (B, shape.heads, shape.value_dim))
        views = [_pack_view(t.data_ptr(), 0, *t.stride()[:2]) for t in (q, k, v, out)]
        _check(lstm_linear_attention_step(shape.packed, views[0], views[1], views[2], log_decay.data_ptr(),
                                          _addr(slots), state.shape[0], state.data_ptr(), views[3], on.handle),
               "lstm_linear_attention_step")
    return out


def _width(t, what):
    if t.dim() == 0 or t.shape[-1] == 0:
        raise ValueError(f"{what} must have a last axis")
    return t.shape[-1]


def _rows(t, what):
    """A tensor whose leading axes are evenly spaced rows (copied if they are not), the spacing, and their number."""
    width = _width(t, what)
    if t.is_contiguous():
        return t, width, t.numel() // width
    if t.dim() != 2 or (width > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < width):
        return t.contiguous(), width, t.numel() // width
    return t, max(t.stride(0), width), t.shape[0]


def layer_norm(x, weight=None, bias=None, eps=1e-5, residual=None, stream=None):
    """Layer norm over the last axis of z = x + residual (lstm_layer_norm_forward).

    Returns (y, mean, rstd, z): y and z in x's dtype and shape (z is x itself without a residual), mean and rstd
    float32 over the leading axes; z, mean and rstd are what layer_norm_backward reads."""
    if torch is None:
        _need_torch()
    code = _code(x, "x")
    width = _width(x, "x")
    for t, what in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _dense(t, x, what, (width,))
    if residual is not None:
        _same(residual, x, "residual", x.shape)
    with _On(x.device, stream) as on:
        xr, xs, rows = _rows(x, "x")
        rr, rs = None, width
        if residual is not None:
            rr, rs, _ = _rows(residual, "residual")
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        z = torch.empty_like(y) if residual is not None else x
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        if on.other is not None:
            on.give(y, mean, rstd, z if residual is not None else None)
        _check(lstm_layer_norm_forward(code, xr.data_ptr(), xs, _addr(rr), rs, _addr(weight), _addr(bias), rows,
                                       width, float(eps), y.data_ptr(), z.data_ptr() if residual is not None else None,
                                       mean.data_ptr(), rstd.data_ptr(), on.handle), "lstm_layer_norm_forward")
    return y, mean, rstd, z


def layer_norm_backward(dy, z, mean, rstd, weight=None, dsum=None, stream=None):
    """Gradients (dz, dweight, dbias) of layer_norm() (lstm_layer_norm_backward).

    dz is the gradient of x and of the residual.  dsum: gradient that reaches z from elsewhere, added to dz.
    dweight and dbias are given without a weight too (the gradients of one that is all ones, and of a zero bias)."""
    if torch is None:
        _need_torch()
    code = _code(z, "z")
    width = _width(z, "z")
    _same(dy, z, "dy", z.shape)
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        _dense(t, z, what, z.shape[:-1], torch.float32)
    if weight is not None:
        _dense(weight, z, "weight", (width,))
    if dsum is not None:
        _same(dsum, z, "dsum", z.shape)
    with _On(z.device, stream) as on:
        yr, ys, rows = _rows(dy, "dy")
        zr, zs, _ = _rows(z, "z")
        sr = dsum.contiguous() if dsum is not None else None
        dz = torch.empty_like(z, memory_format=torch.contiguous_format)
        dw = torch.empty(width, dtype=z.dtype, device=z.device)
        db = torch.empty_like(dw)
        nbytes = lstm_layer_norm_backward_workspace_size(rows, width)
        ws = on.scratch(nbytes)
        if on.other is not None:
            on.give(dz, dw, db)
        _check(lstm_layer_norm_backward(code, yr.data_ptr(), ys, zr.data_ptr(), zs, mean.data_ptr(), rstd.data_ptr(),
                                        _addr(weight), _addr(sr), rows, width, dz.data_ptr(), dw.data_ptr(),
                                        db.data_ptr(), _addr(ws), nbytes, on.handle), "lstm_layer_norm_backward")
    return dz, dw, db


def adamw_states(params, bits=32):
    """Zero states for adamw_step: (m, v, scales), lists like params; scales is None for states of 32 bits, else the
    pair of lists of block scales."""
    if torch is None:
        _need_torch()
    if bits not in (8, 32):
        raise ValueError("states have 8 or 32 bits")
    kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
    m, v = ([torch.zeros(p.shape, dtype=kind, device=p.device) for p in params] for _ in range(2))
    if bits == 32:
        return m, v, None
    count = [-(-p.numel() // LSTM_ADAMW_BLOCK) for p in params]
    ms, vs = ([torch.full((n,), 2.0 ** -126, device=p.device) for n, p in zip(count, params)] for _ in range(2))
    return m, v, (ms, vs)


def adamw_step(params, grads, m, v, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, scales=None,
               masters=None, grad_scale=None, seed=0, stream=None):
    """One AdamW step on lists of contiguous tensors of one dtype, in place (lstm_adamw_step).

    m, v, scales: as adamw_states made them.  step counts from 1.  lr and weight_decay: a number, or one for each
    tensor.  masters: None or a list of float32 copies of bf16 parameters (None entries: no copy).
    grad_scale: None or one float32 on the device that every gradient is multiplied by.
    seed: states of 8 bits are rounded by chance with bits from it; give each step another."""
    if torch is None:
        _need_torch()
    n = len(params)
    if n == 0:
        return
    like = params[0]
    code = _code(like, "params")
    bits = 32 if scales is None else 8
    kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
    ms, vs = scales if scales is not None else ([None] * n, [None] * n)
    masters = masters if masters is not None else [None] * n
    lrs = list(lr) if isinstance(lr, (list, tuple)) else [float(lr)] * n
    wds = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [float(weight_decay)] * n
    if any(len(x) != n for x in (grads, m, v, ms, vs, masters, lrs, wds)):
        raise ValueError("every list must have one entry for each parameter")
    device, dtype = like.device, like.dtype
    parts = []
    for p, g, a, b, sa, sb, w, r, d in zip(params, grads, m, v, ms, vs, masters, lrs, wds):
        size = p.shape
        if not (p.dtype == dtype == g.dtype and a.dtype == kind == b.dtype and g.shape == size == a.shape
                and b.shape == size and p.device == device == g.device and a.device == device == b.device
                and p.is_contiguous() and g.is_contiguous() and a.is_contiguous() and b.is_contiguous()):
            raise ValueError(f"params and grads must be contiguous {dtype} tensors on {device}, m and v contiguous "
                             f"{kind} tensors, each of its parameter's shape")
        count = p.numel()
        if bits == 8:
            blocks = (-(-count // LSTM_ADAMW_BLOCK),)
            _dense(sa, like, "scales", blocks, torch.float32)
            _dense(sb, like, "scales", blocks, torch.float32)
        if w is not None:
            _dense(w, like, "masters", size, torch.float32)
        parts.append(_pack_tensor(p.data_ptr(), g.data_ptr(), a.data_ptr(), b.data_ptr(),
                                  0 if sa is None else sa.data_ptr(), 0 if sb is None else sb.data_ptr(),
                                  0 if w is None else w.data_ptr(), count, r, d))
    table = b"".join(parts)
    if grad_scale is not None:
        _dense(grad_scale, like, "grad_scale", grad_scale.shape, torch.float32)
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must be one float32 value on the device")
    with _On(like.device, stream) as on:
        _check(lstm_adamw_step(code, bits, table, n, float(beta1), float(beta2), float(eps), int(step),
                               _addr(grad_scale), int(seed) & 0xFFFFFFFF, on.handle), "lstm_adamw_step")
