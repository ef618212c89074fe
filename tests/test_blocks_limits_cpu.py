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
