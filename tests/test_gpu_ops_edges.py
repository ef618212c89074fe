"""Operators of include/lstm_ops.h on the GPU where they can go wrong: results that lie over inputs, values at the ends
of fp32's range, other streams, and every tile that the launch rules can choose.  Tolerances are bounds on rounding
against the fp64 oracle, as in test_gpu_ops.py."""
import numpy as np
import pytest

import layer_lstm_forward_amd as pkg
from layer_lstm_forward_amd import ops
from oracle import ops as ref
from tests.test_gpu_ops import DEV, La, U16, U32, close, dev, draw, host, la_tol, ln_tol

pytestmark = pytest.mark.gpu


# ------------------------------------------------- results over their inputs
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [100, 1500, 6000, 20011])
def test_layer_norm_results_over_inputs(width, dtype):
    """y over x, sum over the residual or x; dx over dy or dsum: the same bits as in memory of their own."""
    import torch
    rng = np.random.default_rng(width)
    rows, code = 5, pkg.LSTM_BF16 if dtype == "bf16" else pkg.LSTM_F32
    x, res, dy, ds = (dev(draw(rng, (rows, width), dtype), dtype) for _ in range(4))
    w, b = (dev(draw(rng, (width,), dtype), dtype) for _ in range(2))
    stream = torch.cuda.current_stream().cuda_stream

    def forward(x, res, y, total):
        mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        assert ops.lstm_layer_norm_forward(code, x.data_ptr(), width, res.data_ptr(), width, w.data_ptr(),
                                           b.data_ptr(), rows, width, 1e-5, y.data_ptr(), total.data_ptr(),
                                           mean.data_ptr(), rstd.data_ptr(), stream) == 0
        return y, total, mean, rstd

    print(f"case norm over inputs {rows}x{width} {dtype}", flush=True)
    want = forward(x, res, torch.empty_like(x), torch.empty_like(x))
    for y_over, sum_over in (("x", None), (None, "res"), (None, "x"), ("x", "res")):
        t = {"x": x.clone(), "res": res.clone()}
        got = forward(t["x"], t["res"], t[y_over] if y_over else torch.empty_like(x),
                      t[sum_over] if sum_over else torch.empty_like(x))
        assert all(torch.equal(p, q) for p, q in zip(want, got)), (y_over, sum_over)

    _, z, mean, rstd = want
    nbytes = ops.lstm_layer_norm_backward_workspace_size(rows, width)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)

    def backward(dy, ds, dx):
        dw, db = torch.empty_like(w), torch.empty_like(w)
        assert ops.lstm_layer_norm_backward(code, dy.data_ptr(), width, z.data_ptr(), width, mean.data_ptr(),
                                            rstd.data_ptr(), w.data_ptr(), ds.data_ptr(), rows, width, dx.data_ptr(),
                                            dw.data_ptr(), db.data_ptr(), ws.data_ptr(), nbytes, stream) == 0
        return dx, dw, db

    want = backward(dy, ds, torch.empty_like(dy))
    for over in (0, 1):
        t = [dy.clone(), ds.clone()]
        for p, q, what in zip(want, backward(t[0], t[1], t[over]), ("dx", "dweight", "dbias")):
            assert torch.equal(p, q), (what, "over", ("dy", "dsum")[over])
