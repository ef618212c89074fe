"""Host checks of include/lstm_ops.h at the ends of what the arguments can hold, without a GPU."""
import ctypes
import os

import pytest

import layer_lstm_forward_amd as pkg
from layer_lstm_forward_amd import ops

pytestmark = pytest.mark.skipif(not os.path.exists(pkg.LIB_PATH), reason="liblstm_amd.so not built")

FAKE = 0x10000  # never dereferenced: every case below fails a host check first
MOST_TOKENS = 2 ** 31 - 1 - 2 ** 15


def _shape(**kw):
    a = dict(dtype=1, T=5, B=1, heads=1, kv_heads=1, key_dim=1, value_dim=1, scale=1.0)
    a.update(kw)
    return ops.lstm_linear_attention_shape(**a)


def _v():
    return ops.lstm_view(FAKE, 1, 1, 1)


@pytest.mark.parametrize("T,code", [(MOST_TOKENS, 0), (MOST_TOKENS + 1, -2), (2 ** 31 - 32, -2), (2 ** 31 - 1, -2)])
def test_token_count(T, code):
    """Positions are 32-bit: chunks, segments and the loads ahead of them have to end below 2^31."""
    lib, n = ops._lib(), ctypes.c_size_t()
    s = _shape(T=T)
    assert lib.lstm_linear_attention_workspace_size(s, n) == code
    assert lib.lstm_linear_attention_backward_workspace_size(s, n) == code
    # good but for the memory, which is not on a device
    code = code or -4
    assert ops.lstm_linear_attention_forward(s, _v(), _v(), _v(), FAKE, 0, 0, _v(), 0, FAKE, 1 << 50, 0) == code
    assert ops.lstm_linear_attention_backward(s, _v(), _v(), _v(), FAKE, 0, 0, _v(), 0, _v(), _v(), _v(), 0, FAKE,
                                              1 << 50, 0) == code
