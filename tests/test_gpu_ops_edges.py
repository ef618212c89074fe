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


# ------------------------------------------------------------ other streams
def _busy():
    """Some milliseconds of work queued on the current stream."""
    import torch
    torch.cuda._sleep(20_000_000)


def test_copies_on_another_stream_come_after_their_source():
    """Rows that are not evenly spaced are copied: after the work that is queued on the call's stream."""
    import torch
    rng = np.random.default_rng(31)
    x, res, dy, ds = (dev(draw(rng, (40, 6, 500), "f32")) for _ in range(4))
    w = dev(draw(rng, (500,), "f32"))
    cut = lambda t: t.transpose(0, 1)  # noqa: E731
    y, mean, rstd, z = pkg.layer_norm(cut(x), w, residual=cut(res))
    want = [y, z, *pkg.layer_norm_backward(cut(dy), cut(x), mean, rstd, w, dsum=cut(ds))]
    bufs = [torch.zeros_like(t) for t in (x, res, dy, ds)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _busy()
        for b, t in zip(bufs, (x, res, dy, ds)):
            b.copy_(t)
    bx, bres, bdy, bds = (cut(b) for b in bufs)
    y, _, _, z = pkg.layer_norm(bx, w, residual=bres, stream=side.cuda_stream)
    got = [y, z, *pkg.layer_norm_backward(bdy, bx, mean, rstd, w, dsum=bds, stream=side.cuda_stream)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_memory_on_another_stream_is_free_there():
    """Tensors that were dropped while the current stream still reads them are not written by a call on another."""
    import torch
    c = La(T=2000, B=1, H=2, G=1, Dk=64, Dv=64, dtype="bf16")  # in segments, with a workspace
    rng = np.random.default_rng(32)
    x = dev(draw(rng, (3000, 500), "f32"))
    want = [*c.forward(), *c.backward(), *pkg.layer_norm(x)[:3]]
    dropped = [torch.full_like(t, i + 1.0) for i, t in enumerate(want) for _ in range(3)]
    n = ops.lstm_linear_attention_backward_workspace_size(
        ops.lstm_linear_attention_shape(1, 2000, 1, 2, 1, 64, 64, 0.125))
    dropped += [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for _ in range(3)]
    copies = [torch.empty_like(t) for t in dropped]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy()
    for a, b in zip(copies, dropped):
        a.copy_(b)
    values = [i + 1.0 for i in range(len(want)) for _ in range(3)] + [7] * 3
    del dropped, b
    got = [*c.forward(stream=side.cuda_stream), *c.backward(stream=side.cuda_stream),
           *pkg.layer_norm(x, stream=side.cuda_stream)[:3]]
    torch.cuda.synchronize()
    for t, value in zip(copies, values):
        assert bool((t == value).all())
    for a, b in zip(want, got):
        assert torch.equal(a, b)


# ---------------------------------------------------- the ends of fp32's range
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [("f32", False), ("bf16", False), ("bf16", True)])
def test_adamw_second_moment_overflows(dtype, master, bits):
    """|g| = 1e20: g^2 is infinite in fp32, m is finite, so the step is m / inf = 0, then and in later steps."""
    import torch
    rng = np.random.default_rng(21)
    p = draw(rng, (700,), dtype)
    g = draw(rng, (700,), dtype, 1e-2)
    bad = [5, 256, 511, 699]
    g[bad] = np.float32(1e20)
    tp, lr, wd = [dev(p, dtype)], 1e-2, 0.1
    masters = [dev(p)] if master else None
    m, v, scales = pkg.adamw_states(tp, bits=bits)
    want = p[bad].astype(np.float64)
    tol = np.zeros(len(bad))
    for t in (1, 2, 3):
        pkg.adamw_step(tp, [dev(g if t == 1 else g * 0, dtype)], m, v, step=t, lr=lr, weight_decay=wd, scales=scales,
                       masters=masters, seed=t)
        want *= 1 - lr * wd
        # 1 - lr wd and its product: three roundings; a stored bf16 one more
        tol += (4 * U32 + (U16 if dtype == "bf16" and not master else 0)) * np.abs(want)
        close((masters or tp)[0][bad], want, tol, f"param after step {t}")
    assert bool(torch.isfinite(tp[0]).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [1e-46, 1e-40, 1e-38])
def test_adamw_eps_below_the_normal_range(eps, dtype, bits):
    """Elements that never had a gradient stay: their step is 0 / eps = 0 for every eps above 0."""
    import torch
    p = dev(draw(np.random.default_rng(22), (300,), dtype), dtype)
    old = p.clone()
    m, v, scales = pkg.adamw_states([p], bits=bits)
    for t in (1, 2):
        pkg.adamw_step([p], [torch.zeros_like(p)], m, v, step=t, eps=eps, weight_decay=0.0, scales=scales, seed=t)
    assert torch.equal(p, old)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_attention_growing_state(dtype):
    """gamma above 1.  The first tokens have zero keys, so that the state stays small although gamma^T leaves the fp32
    range."""
    c = La(T=140, B=2, H=4, G=4, Dk=20, Dv=24, dtype=dtype, decays=[1.0, 0.3, 0.12, 0.05], state=False)
    c.k[:, :80] = 0
    c.tk = dev(c.seq(c.k), dtype)
    c.check_forward(c.forward())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale,size", [(1e-30, 1e10), (1e-39, 1.0), (1e25, 1e-10)])
def test_linear_attention_gradients_at_any_scale(scale, size, dtype):
    """The gradient of the state does not depend on the scale: a row of no tokens passes it on as it is."""
    import torch
    c = La(T=50, B=3, H=2, G=1, Dk=32, Dv=40, dtype=dtype, lengths=[50, 0, 33], scale=scale)
    c.dS = c.dS * np.float32(size)
    c.tdS = dev(c.dS)
    grads = c.backward()
    c.check_backward(grads)
    assert torch.equal(grads[3][1], c.tdS[1])


def test_layer_norm_gradient_of_a_large_constant_row():
    """The variance is 0 and mean * rstd leaves the fp32 range; the row's own values are all 0 after the norm."""
    rng = np.random.default_rng(23)
    z, dy = np.full((3, 8), 1e37, np.float32), draw(rng, (3, 8), "f32")
    z[1] = draw(rng, (8,), "f32")
    y, mean, rstd, total = pkg.layer_norm(dev(z))
    dz, dw, db = pkg.layer_norm_backward(dev(dy), total, mean, rstd)
    wz, wdw, wdb = ref.layer_norm_backward(dy, z.astype(np.float64))
    wr = ref.layer_norm(z.astype(np.float64))[2][:, None]
    close(dz, wz, 64 * U32 * wr * (np.abs(dy) + np.abs(dy).mean(1, keepdims=True)) * 8, "dz")
    close(dw, wdw, 64 * U32 * 8 * np.abs(dy).sum(0), "dweight")
    close(db, wdb, 8 * U32 * np.abs(dy).sum(0), "dbias")
