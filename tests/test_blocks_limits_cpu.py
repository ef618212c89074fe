"""Arguments of the wrappers of include/lstm_blocks.h at the ends of what they can hold, without a GPU."""
import pytest

import layer_lstm_forward_amd as pkg
from tests.test_blocks_cpu import kernels  # noqa: F401  (a fixture)
from tests.test_ops_streams_cpu import NOTES, device, put  # noqa: F401  (device: a fixture)


@pytest.mark.parametrize("kw", [dict(eps=1e-50), dict(eps=1e39), dict(scale=1e39), dict(scale=-1e39), dict(scale=1e-60)])
def test_rotary_numbers_outside_fp32(kernels, kw):  # noqa: F811
    """An eps that fp32 does not hold would be 0, and a row of zeros not a number."""
    import torch
    q = put(5, 2, 4, 8)
    f = torch.zeros(4, dtype=torch.float64).as_subclass(type(q))
    with pytest.raises(ValueError):
        pkg.rotary(q, None, f, norm=True, **kw)
    with pytest.raises(ValueError):
        pkg.rotary_backward(q, None, f, q, None, norm=True, **kw)
    assert not [n for n in NOTES if n[0] == "kernels"]
    pkg.rotary(q, None, f, norm=True, eps=0.0, scale=1e-40)
    pkg.rotary(q, None, f, norm=True, eps=1e-45, scale=0.0)


def test_expanded_outputs(kernels):  # noqa: F811
    """A tensor whose elements share memory is no place to write to."""
    import torch
    x, S = put(5, 2, 8), put(2, 8)
    q, f = put(5, 2, 4, 8), torch.zeros(4, dtype=torch.float64).as_subclass(type(x))
    flat, wide = put(1, 2, 8).expand(5, 2, 8), put(5, 2, 1, 8).expand(5, 2, 4, 8)
    for call in (
            lambda: pkg.gated_recurrence(x, x, out=(flat, S)),
            lambda: pkg.gated_recurrence_backward(x, x, x, x, out=(flat, x, None)),
            lambda: pkg.gated_recurrence_backward(x, x, x, x, out=(x, flat, None)),
            lambda: pkg.gated_recurrence_backward(x, x, x, x, input_gate=x, out=(x, x, flat)),
            lambda: pkg.gated_recurrence_step(x[0], x[0], S, out=put(1, 8).expand(2, 8)),
            lambda: pkg.rotary(q, q, f, out=(wide, q)), lambda: pkg.rotary(q, q, f, out=(q, wide)),
            lambda: pkg.rotary_backward(q, q, f, q, q, out=(wide, q)),
            lambda: pkg.rotary_backward(q, q, f, q, q, out=(q, wide))):
        with pytest.raises(ValueError):
            call()
    assert not [n for n in NOTES if n[0] == "kernels"]
    one = put(1, 2, 8).expand(1, 2, 8)  # (an axis of one has any stride)
    pkg.gated_recurrence(one, one, out=(one.as_strided((1, 2, 8), (0, 8, 1)), S))
    pkg.rotary(wide, flat[..., None, :], f, out=(q, put(5, 2, 1, 8)))  # inputs may repeat


def test_keys_of_no_heads(kernels, monkeypatch):  # noqa: F811
    """The gradient of a weight that nothing reads is 0, not what its memory held."""
    import torch
    q = put(5, 2, 4, 8)
    f, w = torch.zeros(4, dtype=torch.float64).as_subclass(type(q)), put(8)
    monkeypatch.setattr(type(q), "new_empty", lambda t, *a: torch.full(a[0] if isinstance(a[0], tuple) else a, 7.0,
                                                                       dtype=t.dtype).as_subclass(type(q)))
    dwk = pkg.rotary_backward(q, q[:, :, :0], f, q, q[:, :, :0], q_weight=w, k_weight=w, norm=True)[3]
    assert not dwk.any()
