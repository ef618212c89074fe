"""Operators of include/lstm_ops.h on the GPU where they can go wrong: results that lie over inputs, values at the ends
of fp32's range, other streams, and every tile that the launch rules can choose.  Tolerances are bounds on rounding
against the fp64 oracle, as in test_gpu_ops.py."""
import numpy as np
import pytest

import layer_lstm_forward_amd as pkg
from layer_lstm_forward_amd import ops
from oracle import ops as ref
from tests.test_gpu_ops import DEV, La, U16, U32, close, dev, draw, host, ln_tol

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


# ------------------------------------- every tile that the launch rules choose
# (batch row, head) pairs, doubled or tripled by passes, and dims decide; see la_plan
TILES = {
    # two column tiles a wave, half of each width: above 192 pairs, or above 1024 tokens
    "pairs-direct": dict(T=70, B=50, H=4, G=2, Dk=128, Dv=128, packed=True,
                         lengths=[70, 0, 1, 31, 32, 33, 64, 65, 69] + [70] * 41),
    "long-direct": dict(T=1100, B=1, H=2, G=1, Dk=128, Dv=128, decays=[-0.2, -0.001]),
    "long-direct-ragged": dict(T=1060, B=2, H=1, G=1, Dk=128, Dv=128, lengths=[700, 1060], batch_first=True),
    "pairs-edges": dict(T=45, B=50, H=4, G=2, Dk=72, Dv=104, packed=True, lengths=[45, 0, 1, 32, 33] + [45] * 45),
    "pairs-short": dict(T=40, B=50, H=4, G=4, Dk=100, Dv=3),
    # eight waves for fp32: above 128 pairs and values wider than 64
    "eight-64": dict(T=70, B=33, H=4, G=2, Dk=64, Dv=128, lengths=[70, 0, 1, 31, 32, 33, 64, 65] + [70] * 25),
    "eight-64-odd": dict(T=40, B=66, H=2, G=1, Dk=50, Dv=90, packed=True),
    "eight-128-odd": dict(T=40, B=33, H=4, G=1, Dk=101, Dv=127, packed=True, batch_first=True),
    "eight-short": dict(T=40, B=33, H=4, G=4, Dk=3, Dv=100),
    "eight-256": dict(T=35, B=65, H=2, G=2, Dk=256, Dv=256, lengths=[35, 0, 1, 32, 33] + [35] * 60),
    "eight-256-odd": dict(T=35, B=65, H=2, G=1, Dk=200, Dv=250),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", TILES)
def test_linear_attention_tiles(name, dtype):
    c = La(dtype=dtype, **TILES[name])
    print(f"case {name} {dtype} forward", flush=True)
    c.check_forward(c.forward())
    print(f"case {name} {dtype} backward", flush=True)
    c.check_backward(c.backward())


@pytest.mark.parametrize("B,H", [(1, 2), (50, 4)])
def test_linear_attention_state_keeps_fp32_products(B, H):
    """A state that is returned is summed from bf16 operands as if their weighted products were fp32.  Two of the three
    bf16 terms that a weighted value is split into would leave 2^-17 of it (an rms of about 2.7e-6); fp32 sums of 400
    terms in chunks of 32 stay near 2^-22."""
    c = La(T=400, B=B, H=H, G=H, Dk=128, Dv=128, dtype="bf16", decays=[-0.002 * (h + 1) for h in range(H)])
    few = [0, B - 1]
    got, grad = host(c.forward()[1])[few], host(c.backward()[3])[few]
    a = [x[few] for x in (c.q, c.k, c.v, c.do, c.S, c.dS)]
    want = ref.linear_attention(a[0], a[1], a[2], c.g, c.scale, a[4])[1]
    wgrad = ref.linear_attention_backward(a[0], a[1], a[2], c.g, c.scale, a[3], a[4], a[5])[3]
    for x, w, what in ((got, want, "state"), (grad, wgrad, "dstate")):
        off = np.sqrt(((x - w) ** 2).mean() / (w ** 2).mean())
        assert off < 1e-6, (what, off)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,G,Dk,Dv", [(130, 4, 2, 40, 72), (260, 2, 2, 200, 128), (520, 1, 1, 16, 36),
                                         (6, 2, 1, 200, 33), (300, 2, 2, 150, 30)])
def test_linear_attention_step_tiles(B, H, G, Dk, Dv, dtype):
    """512 states and more take wider column slabs; rows past the first 128 are a second round there."""
    rng = np.random.default_rng(B + Dv)
    q, k = draw(rng, (B, 1, H, Dk), dtype), draw(rng, (B, 1, G, Dk), dtype)
    v, g = draw(rng, (B, 1, G, Dv), dtype), -rng.uniform(0, 2, H).astype(np.float32)
    slots = rng.permutation(B + 3)[:B].astype(np.int32)
    slots[1] = -1
    busy = slots >= 0
    pool = draw(rng, (B + 3, H, Dk, Dv), "f32")
    at = np.where(busy, slots, 0)
    wo, ws = ref.linear_attention(q, k, v, g, Dk ** -0.5, pool[at])
    Ao, As = ref.linear_attention(np.abs(q), np.abs(k), np.abs(v), g, Dk ** -0.5, np.abs(pool[at]))
    tp = dev(pool)
    o = pkg.linear_attention_step(*(dev(x[:, 0], dtype) for x in (q, k, v)), dev(g), tp, slots=dev(slots))
    want, tol = pool.astype(np.float64), np.zeros(pool.shape)
    want[slots[busy]], tol[slots[busy]] = ws[busy], 4 * U32 * As[busy] + 1e-30
    close(tp, want, tol, "pool")
    wo = np.where(busy[:, None, None, None], wo, 0.0)
    close(o, wo[:, 0], ((Dk + 8) * U32 * Ao + (U16 * np.abs(wo) if dtype == "bf16" else 0) + 1e-30)[:, 0], "o")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(9, 1025), (700, 1536), (5, 2048), (6, 2047), (530, 2048), (5, 2049),
                                        (260, 6001)])
def test_layer_norm_tiles(rows, width, dtype):
    rng = np.random.default_rng(rows + width)
    x, res, dy, ds = (draw(rng, (rows, width), dtype) for _ in range(4))
    w, b = draw(rng, (width,), dtype), draw(rng, (width,), dtype)
    t = lambda a: dev(a, dtype)  # noqa: E731
    y, mean, rstd, total = pkg.layer_norm(t(x), t(w), t(b), residual=t(res))
    z = host(total)
    half = U16 if dtype == "bf16" else 2 * U32
    close(total, x.astype(np.float64) + res, half * np.abs(x.astype(np.float64) + res), "sum")
    wy, wm, wr = ref.layer_norm(z, w, b)
    unit = (z - wm[:, None]) * wr[:, None]
    tol, rel = ln_tol(z, w.astype(np.float64), unit, wr, dtype)
    close(y, wy, tol + half * np.abs(wy) + 4 * U32 * np.abs(b.astype(np.float64)) + half * 1e-30, "y")
    close(mean, wm, (width / 64 + 16) * U32 * np.abs(z).mean(1) + 1e-30, "mean")
    close(rstd, wr, rel * wr, "rstd")
    dz, dw, db = pkg.layer_norm_backward(t(dy), total, mean, rstd, t(w), dsum=t(ds))
    wz, wdw, wdb = ref.layer_norm_backward(dy, z, w, dsum=ds)
    g = np.abs(dy.astype(np.float64) * w)
    A = wr[:, None] * (g + g.mean(1, keepdims=True)
                       + (np.abs(unit) + 1) * (g * (np.abs(unit) + 1)).mean(1, keepdims=True))
    close(dz, wz, 4 * rel[:, None] * A + 4 * U32 * np.abs(ds) + half * np.abs(wz), "dz")
    close(dw, wdw, (np.abs(dy) * (np.abs(unit) + 1) * (2 * rel + rows * U32)[:, None]).sum(0) + half * np.abs(wdw),
          "dweight")
    close(db, wdb, (rows + 4) * U32 * np.abs(dy.astype(np.float64)).sum(0) + half * np.abs(wdb), "dbias")


@pytest.mark.parametrize("dtype,master,bits", [("bf16", False, 32), ("bf16", True, 32), ("f32", False, 8),
                                               ("bf16", False, 8), ("bf16", True, 8)])
def test_adamw_large_lists(dtype, master, bits):
    """2^23 elements and more take four pieces a thread: whole ones, a tensor's end, and one that starts at an odd
    element."""
    import torch
    rng = np.random.default_rng(24)
    shapes = [((1 << 23) + 777, 0), (5000, 0), (20001, 1)]
    p, g = [draw(rng, (n,), dtype) for n, _ in shapes], [draw(rng, (n,), dtype, 1e-2) for n, _ in shapes]

    def put(a, dt, off):
        t = torch.empty(a.size + off, dtype=torch.bfloat16 if dt == "bf16" else torch.float32, device=DEV)[off:]
        t.copy_(dev(a, dt))
        return t

    tp, tg = ([put(a, dtype, off) for a, (_, off) in zip(x, shapes)] for x in (p, g))
    masters = [put(a, "f32", off) for a, (_, off) in zip(p, shapes)] if master else None
    m, v, scales = pkg.adamw_states(tp, bits=bits)
    pkg.adamw_step(tp, tg, m, v, step=1, lr=1e-2, scales=scales, masters=masters, seed=5)
    values = ref.code_values()
    for i, (a, b) in enumerate(zip(p, g)):
        wp, wm, wv = ref.adamw(a, b, 0.0, 0.0, 1, 1e-2, 0.9, 0.999, 1e-8, 0.01)
        step = np.abs(1e-2 * (wm / (1 - 0.9)) / (np.sqrt(wv / (1 - 0.999)) + 1e-8))
        tol = 16 * U32 * (np.abs(wp) + 4 * step)
        if master:
            close(masters[i], wp, tol, "master")
            assert torch.equal(masters[i].to(torch.bfloat16), tp[i])
        else:
            close(tp[i], wp, tol + (U16 * np.abs(wp) if dtype == "bf16" else 0), "param")
        if bits == 32:
            close(m[i], wm, 16 * U32 * np.abs(wm), "m")
            close(v[i], wv, 24 * U32 * np.abs(wv), "v")
            continue
        for got, sc, want in ((m[i], scales[0][i], wm), (v[i], scales[1][i], np.sqrt(wv))):
            top = np.maximum.reduceat(np.abs(want), np.arange(0, want.size, 256))
            assert np.array_equal(host(sc), np.exp2(np.maximum(np.floor(np.log2(np.maximum(top, 1e-300))) - 7, -126.0)))
            s = np.repeat(host(sc), 256)[:want.size]
            x = values[got.view(torch.uint8).cpu().numpy()] * s
            unit = np.exp2(np.floor(np.log2(np.maximum(np.abs(want) / s, 2.0 ** -6))) - 3) * s
            assert np.all(np.abs(x - want) <= unit * (1 + 1e-4))


def test_layer_norm_widest_rows():
    """2^28 values, the limit: one row, and its weight gradients."""
    import torch
    width = 1 << 28
    gen = torch.Generator(device=DEV)
    gen.manual_seed(25)
    x, dy = (torch.randn(1, width, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    y, mean, rstd, z = pkg.layer_norm(x)
    dz, dw, db = pkg.layer_norm_backward(dy, z, mean, rstd)
    m = x.double().mean()
    # chains of 2^20 additions: of values of both signs they wander, by about the root of their number
    assert abs(float(mean[0]) - float(m)) < 2 ** 10 * 24 * U32
    assert abs(float(rstd[0]) - float((x.double() - m).square().mean() + 1e-5) ** -0.5) < 1e-3
    unit = (x.float() - mean) * rstd
    for a, b, what in ((y[0], unit[0], "y"), (dw, (dy.float() * unit)[0], "dweight"), (db, dy[0].float(), "dbias")):
        # the statistics are the kernel's own: three roundings and the result's
        assert bool(((a.float() - b).abs() <= (U16 + 4 * U32) * b.abs() + 1e-30).all()), what
    g = dy.float()
    want = rstd * (g - g.double().mean().float() - unit * (g * unit).double().mean().float())
    assert bool(((dz.float() - want).abs() <= 2 * U16 * want.abs() + 1e-3).all())


def test_refusals_of_empty_axes():
    import torch
    one = torch.ones((), device=DEV)
    with pytest.raises(ValueError):
        pkg.layer_norm(one)
    with pytest.raises(ValueError):
        pkg.layer_norm_backward(one, one, one, one)
    for shape in ((3, 0), (0,)):
        x = torch.ones(shape, device=DEV)
        with pytest.raises(ValueError):
            pkg.layer_norm(x)
    g = torch.zeros(2, device=DEV)
    for T, B, H, D in ((0, 1, 2, 8), (3, 0, 2, 8), (3, 1, 2, 0)):
        q, S = torch.ones(T, B, H, D, device=DEV), torch.ones(B, H, D, D, device=DEV)
        for scale in (None, 1.0):
            with pytest.raises((ValueError, pkg.LSTMError)):
                pkg.linear_attention(q, q, q, g, scale=scale)
            with pytest.raises((ValueError, pkg.LSTMError)):
                pkg.linear_attention_backward(q, q, q, g, q, scale=scale)
            if T:
                with pytest.raises((ValueError, pkg.LSTMError)):
                    pkg.linear_attention_step(q[0], q[0], q[0], g, S, scale=scale)
