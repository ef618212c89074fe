"""The operators of include/lstm_blocks.h on the GPU against the fp64 oracle.

Tolerances are bounds on rounding, element by element, carried through the same formulas as the values: U32 and U16
are half a step of fp32 and bf16, and every fp32 operation, hardware exponential or reciprocal costs a few U32 of what
it works on.
"""
import numpy as np
import pytest

import layer_lstm_forward_amd as pkg
from oracle import blocks as ref
from tests.test_gpu_ops import DEV, U16, U32, close, dev, draw, host

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------- gated recurrence
class Rec:
    """Inputs of a case; host copies are exact in the dtype, [B, T, W]."""

    def __init__(self, T, B, W, dtype, gates=1, state=True, lengths=None, batch_first=False, packed=False, keep=2.0,
                 seed=0):
        rng = np.random.default_rng(seed + 31 * T + W)
        self.__dict__.update(T=T, B=B, W=W, dtype=dtype, batch_first=batch_first, lengths=lengths, packed=packed)
        self.x, self.dy = draw(rng, (B, T, W), dtype), draw(rng, (B, T, W), dtype)
        f = draw(rng, (B, T, W), "f32") + np.linspace(0, keep, W, dtype=np.float32)
        self.f = host(dev(f, dtype)).astype(np.float32)
        self.i = draw(rng, (B, T, W), dtype) if gates == 2 else None
        self.S = draw(rng, (B, W), "f32") if state else None
        self.dS = draw(rng, (B, W), "f32") if state else None

    def tensors(self):
        """x, forget, input gate and dy on the device, what is past a row's end not a number."""
        arrays = [self.x, self.f] + ([self.i] if self.i is not None else []) + [self.dy]
        if self.lengths is not None:
            arrays = [a.copy() for a in arrays]
            for a in arrays:
                for b, n in enumerate(self.lengths):
                    a[b, n:] = np.nan
        if not self.batch_first:
            arrays = [a.transpose(1, 0, 2) for a in arrays]
        if self.packed:
            wide = dev(np.concatenate(arrays, -1), self.dtype)
            out = list(wide.split(self.W, -1))
        else:
            out = [dev(a, self.dtype) for a in arrays]
        if self.i is None:
            out.insert(2, None)
        return out

    def host(self, t):
        a = host(t)
        return a if self.batch_first else a.transpose(1, 0, 2)

    def bounds(self):
        """Errors of y, the state, dx, df, di and dstate.  A step: the gates are off by (8 + 2 |logit|) U32 (the
        exponent's rounding moves the exponential by the logit's size), the sum by 4 U32 of its parts; segments of a
        long sequence carry the product of their gates, which is another 2 U32 a step of what it multiplies."""
        B, T, W = self.x.shape
        f, x = self.f.astype(np.float64), np.abs(self.x.astype(np.float64))
        a, z = ref.logistic(f), ref.logistic(-f)
        cf = (8 + 2 * np.abs(f)) * U32
        w, cw = (z, cf) if self.i is None else (ref.logistic(self.i), (8 + 2 * np.abs(self.i)) * U32)
        rough = U16 if self.dtype == "bf16" else 0.0
        n = [T] * B if self.lengths is None else self.lengths
        ey, es, mag = np.zeros((B, T, W)), np.zeros((B, W)), np.zeros((B, T + 1, W))
        eh = np.zeros((B, T + 1, W))
        ex, ef, ei, eds = np.zeros((B, T, W)), np.zeros((B, T, W)), np.zeros((B, T, W)), np.zeros((B, W))
        for b in range(B):
            h = np.zeros(W) if self.S is None else np.abs(self.S[b].astype(np.float64))
            e = np.zeros(W)
            mag[b, 0] = h
            for t in range(n[b]):
                e = a[b, t] * e + cf[b, t] * z[b, t] * h + cw[b, t] * w[b, t] * x[b, t]
                h = a[b, t] * h + w[b, t] * x[b, t]
                e = e + 6 * U32 * h
                ey[b, t], eh[b, t + 1], mag[b, t + 1] = e + rough * h, e, h
            es[b] = e
            D = np.zeros(W) if self.dS is None else np.abs(self.dS[b].astype(np.float64))
            e = np.zeros(W)
            for t in range(n[b] - 1, -1, -1):
                D = D + np.abs(self.dy[b, t])
                e = e + 4 * U32 * D
                was = mag[b, t] + (x[b, t] if self.i is None else 0.0)
                off = eh[b, t] + (rough * mag[b, t] if t else 0.0) + 2 * U32 * was
                s = a[b, t] * z[b, t]
                ex[b, t] = w[b, t] * (e + (cw[b, t] + 2 * U32) * D)
                ef[b, t] = s * (e * was + D * off + (2 * cf[b, t] + 6 * U32) * D * was)
                if self.i is not None:
                    v = w[b, t] * (1 - w[b, t])
                    ei[b, t] = v * x[b, t] * (e + (2 * cw[b, t] + 6 * U32) * D)
                if rough:
                    ex[b, t] += rough * w[b, t] * D
                    ef[b, t] += rough * s * D * was
                    ei[b, t] += rough * w[b, t] * (1 - w[b, t]) * x[b, t] * D
                e = a[b, t] * e + (cf[b, t] * z[b, t] + 6 * U32) * D
                D = a[b, t] * D
            eds[b] = e
        return [v + 1e-30 for v in (ey, es, ex, ef, ei, eds)]

    def check(self):
        x, f, i, dy = self.tensors()
        more = dict(input_gate=i, state=None if self.S is None else dev(self.S), lengths=self.lengths,
                    batch_first=self.batch_first)
        y, last = pkg.gated_recurrence(x, f, **more)
        dS = None if self.dS is None else dev(self.dS)
        dx, df, di, dstate = pkg.gated_recurrence_backward(x, f, y, dy, dstate=dS, **more)
        ry, rlast = ref.gated_recurrence(self.x, self.f, self.i, self.S, self.lengths)
        rx, rf, ri, rs = ref.gated_recurrence_backward(self.x, self.f, self.dy, self.i, self.S, self.dS, self.lengths)
        ey, es, ex, ef, ei, eds = self.bounds()
        for got, want, tol, what in ((y, ry, ey, "y"), (dx, rx, ex, "dx"), (df, rf, ef, "dforget"), (di, ri, ei, "di")):
            if got is not None:
                close(dev(self.host(got)), want, tol, what)
        close(last, rlast, es, "state")
        if self.S is not None:
            close(dstate, rs, eds, "dstate")
        if self.lengths is not None:
            for t in (y, dx, df):
                for b, n in enumerate(self.lengths):
                    assert not self.host(t)[b, n:].any()
        return y, last


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,W,gates", [(1, 1, 1, 1), (1, 3, 16, 2), (2, 1, 7, 1), (9, 2, 8, 2), (33, 3, 65, 1),
                                         (64, 2, 512, 2), (129, 1, 1001, 1), (700, 2, 24, 2), (2048, 1, 40, 1)])
def test_recurrence(T, B, W, gates, dtype):
    Rec(T, B, W, dtype, gates).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch_first,packed,state", [(True, True, True), (False, True, False), (True, False, False)])
def test_recurrence_layouts(batch_first, packed, state, dtype):
    Rec(75, 4, 37, dtype, 2, state=state, batch_first=batch_first, packed=packed).check()
    Rec(75, 4, 37, dtype, 1, state=state, batch_first=batch_first, packed=packed, lengths=[0, 75, 1, 40]).check()


@pytest.mark.parametrize("T", [40, 1000])
def test_recurrence_lengths(T):
    Rec(T, 6, 20, "f32", 2, lengths=[T, 0, 1, T - 1, 33, T // 2]).check()
    Rec(T, 3, 20, "bf16", 1, lengths=[0, 0, 0]).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,W,gates", [(11, 300, 1000, 1), (11, 290, 1003, 2), (40, 150, 515, 1)])
def test_recurrence_many_channels(T, B, W, gates, dtype):
    """Enough channels for the card without cutting the sequence; rows of every length."""
    Rec(T, B, W, dtype, gates, lengths=[b % (T + 1) for b in range(B)], packed=gates == 2).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,W,gates", [(1500, 2, 9, 1), (3000, 1, 130, 2), (4097, 1, 3, 1), (1025, 5, 67, 2)])
def test_recurrence_in_a_chain(T, B, W, gates, dtype):
    """Few channels and many tokens: tiles that hand their carries on, rows that end in the first, inside and at the end
    of one, or have none."""
    Rec(T, B, W, dtype, gates, lengths=[T, T - 700, 0, 128, 3][:B]).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,W,gates", [(1500, 2, 9, 1), (3000, 1, 130, 2), (4097, 1, 3, 1)])
def test_recurrence_in_segments(T, B, W, gates, dtype):
    Rec(T, B, W, dtype, gates, lengths=[T] if B == 1 else [T - 700, T]).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_recurrence_chain_gives_the_same_bits(dtype):
    """Which of the tiles before it a tile finds first is a matter of time; the results are not."""
    import torch
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, f, dy = (torch.randn(9000, 1, 200, generator=gen, device=DEV).to(dt) for _ in range(3))
    f += 3
    want = None
    for _ in range(5):
        y, last = pkg.gated_recurrence(x, f)
        got = [y, last, *pkg.gated_recurrence_backward(x, f, y, dy)[:2]]
        assert want is None or all(torch.equal(a, b) for a, b in zip(want, got))
        want = got


@pytest.mark.parametrize("T,B,W", [(40, 2, 24), (1500, 1, 24), (11, 300, 1000)])
def test_recurrence_not_finite_and_saturated(T, B, W):
    """A token that is not a number reaches its channel's later tokens alone; gates at both ends keep and take exactly."""
    import torch
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    x, f = (torch.randn(T, B, W, generator=gen, device=DEV) for _ in range(2))
    want, _ = pkg.gated_recurrence(x, f)
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[T // 2, 0, 5] = bad
        got, _ = pkg.gated_recurrence(z, f)
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[T // 2:, 0, 5] = True
        assert torch.equal(got[~hit], want[~hit]) and not torch.isfinite(got[hit]).any()
    S = torch.randn(B, W, generator=gen, device=DEV)
    for logit in (200.0, float("inf")):
        y, last = pkg.gated_recurrence(x, torch.full_like(f, logit), state=S)
        assert torch.equal(y, S.expand_as(y)) and torch.equal(last, S)
        y, last = pkg.gated_recurrence(x, torch.full_like(f, -logit), state=S)
        assert torch.equal(y, x) and torch.equal(last, x[-1])


def test_recurrence_long_memory():
    """Gates so near 1 that 1 - a has no digits left in a itself (logits up to 20)."""
    Rec(512, 2, 64, "f32", 1, keep=20.0).check()


def test_recurrence_state_in_place_and_continued():
    """Two halves, the state updated in place, against the whole, at a width whose last piece overlaps."""
    import torch
    c = Rec(64, 2, 13, "f32", 1)
    x, f, _, _ = c.tensors()
    S = dev(c.S)
    y, last = pkg.gated_recurrence(x, f, state=S)
    half = torch.empty_like(x)
    for k in (0, 32):
        pkg.gated_recurrence(x[k:k + 32], f[k:k + 32], state=S, out=(half[k:k + 32], S))
    ey, es = c.bounds()[:2]
    close(half.transpose(0, 1), host(y).transpose(1, 0, 2), 2 * ey, "y")
    close(S, host(last), 2 * es, "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W,gates", [(1, 1), (30, 2), (64, 1), (1024, 2)])
def test_recurrence_step(W, gates, dtype):
    import torch
    c = Rec(1, 5, W, dtype, gates)
    x, f, i, _ = (None if t is None else t[0] for t in c.tensors())
    pool = np.random.default_rng(3).standard_normal((9, W)).astype(np.float32)
    slots = np.array([8, -1, 0, 9, 4], np.int32)
    state = dev(pool)
    y = pkg.gated_recurrence_step(x, f, state, input_gate=i, slots=torch.from_numpy(slots).to(DEV))
    want, out = pool.astype(np.float64), np.zeros((5, W))
    tol, ty = np.zeros_like(want), np.zeros((5, W))
    for b, s in enumerate(slots):
        if 0 <= s < 9:
            one = Rec.__new__(Rec)
            one.__dict__.update(c.__dict__, x=c.x[b:b + 1], f=c.f[b:b + 1], i=None if i is None else c.i[b:b + 1],
                                dy=c.dy[b:b + 1], S=pool[s:s + 1], dS=None)
            ry, rl = ref.gated_recurrence(one.x, one.f, one.i, one.S)
            ey, es = one.bounds()[:2]
            want[s], out[b], tol[s], ty[b] = rl[0], ry[0, 0], es[0], ey[0, 0]
    close(state, want, tol, "pool")
    close(y, out, ty, "y")
    # without slots row b is state[b]; a sequence of one token does the same
    state = dev(pool[:5])
    y = pkg.gated_recurrence_step(x, f, state, input_gate=i)
    y1, last = pkg.gated_recurrence(x[None], f[None], input_gate=None if i is None else i[None], state=dev(pool[:5]))
    assert torch.equal(y, y1[0]) and torch.equal(state, last)


# -------------------------------------------------------------------- rotary
def rot_case(T, B, H, G, D, rot, dtype, interleaved=False, norm=True, weights=True, far=0, batch_first=False,
             packed=False, scale=1.0, eps=1e-6, seed=0):
    import torch
    rng = np.random.default_rng(seed + T + 7 * D)
    lead = (B, T) if batch_first else (T, B)
    q, k = draw(rng, lead + (H, D), dtype), draw(rng, lead + (G, D), dtype)
    dq, dk = draw(rng, lead + (H, D), dtype), draw(rng, lead + (G, D), dtype)
    w = [draw(rng, (D,), dtype) if norm and weights else None for _ in range(2)]
    freq = pkg.rotary_frequencies(rot, device=DEV)
    pos = rng.integers(-5, far, lead).astype(np.int32) if far else None
    at = pos if pos is not None else np.broadcast_to(np.arange(T)[None] if batch_first else np.arange(T)[:, None], lead)
    if packed:
        wide = dev(np.concatenate([q.reshape(lead + (-1,)), k.reshape(lead + (-1,))], -1), dtype)
        tq, tk = wide[..., :H * D].unflatten(-1, (H, D)), wide[..., H * D:].unflatten(-1, (G, D))
    else:
        tq, tk = dev(q, dtype), dev(k, dtype)
    tw = [None if v is None else dev(v, dtype) for v in w]
    more = dict(positions=None if pos is None else torch.from_numpy(pos).to(DEV), q_weight=tw[0], k_weight=tw[1],
                norm=norm, eps=eps, interleaved=interleaved, scale=scale, batch_first=batch_first)
    a = dict(norm=norm, eps=eps, interleaved=interleaved, scale=scale)
    f = freq.cpu().numpy()
    got = pkg.rotary(tq, tk, freq, **more)
    back = pkg.rotary_backward(tq, tk, freq, dev(dq, dtype), dev(dk, dtype), **more)
    rough = U16 if dtype == "bf16" else 0.0
    m = max(1.0, abs(scale))
    for s, (x, dy, wt) in enumerate(((q, dq, w[0]), (k, dk, w[1]))):
        want = ref.rotary(x, at, f, wt, **a)
        # what a pair holds, and the norm's sum of D squares; sines and cosines to 8 U32
        u = np.abs(ref.rotary(x, np.zeros(lead), f[:0], wt, norm=norm, eps=eps))
        pair = np.broadcast_to(u.max(-1, keepdims=True), u.shape) * 2 * m
        close(got[s], want, (D + 32) * U32 * pair + rough * np.abs(want) + 1e-30, "qk"[s])
        dx, dw = ref.rotary_backward(x, dy, at, f, wt, **a)
        g = np.broadcast_to(np.abs(dy).max(-1, keepdims=True), dy.shape) * 2.0 * m
        if norm:
            x64 = x.astype(np.float64)
            r = 1.0 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + eps)
            unit, v = np.abs(x64 * r), g * (1.0 if wt is None else np.abs(wt))
            size = r * (v + unit * (v * unit).mean(-1, keepdims=True))
            close(back[2 + s], dw, ((T * B * x.shape[2] + 2 * D + 64) * U32 * (g * unit)).reshape(-1, D).sum(0)
                  + rough * np.abs(dw) + 1e-30, "dw")
        else:
            size = g
            assert back[2 + s] is None
        close(back[s], dx, (2 * D + 64) * U32 * size + rough * np.abs(dx) + 1e-30, "d" + "qk"[s])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot", [(1, 0), (2, 2), (9, 6), (16, 16), (40, 20), (64, 64), (72, 40), (128, 128), (127, 50),
                                   (130, 130), (255, 254), (256, 64), (256, 256)])
def test_rotary(D, rot, norm, interleaved, dtype):
    rot_case(5, 3, 3, 2, D, rot, dtype, interleaved, norm)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rotary_layouts(dtype):
    rot_case(1, 1, 1, 1, 64, 64, dtype)
    rot_case(40, 2, 17, 9, 64, 64, dtype, batch_first=True, packed=True, far=1000000)
    rot_case(300, 3, 4, 1, 24, 8, dtype, interleaved=True, packed=True, far=2 ** 31 - 1, weights=False)
    rot_case(7, 5, 8, 16, 128, 64, dtype, scale=1.25, far=200)
    rot_case(3000, 1, 2, 2, 32, 32, dtype)


def test_rotary_without_keys_in_place_and_single_tokens():
    import torch
    freq = pkg.rotary_frequencies(32, device=DEV)
    x = torch.randn(6, 4, 32, device=DEV)
    pos = torch.tensor([3, 1, 4, 1, 5, 9], dtype=torch.int32, device=DEV)
    want, none = pkg.rotary(x[None], None, freq, positions=pos[None], norm=True)
    got, _ = pkg.rotary(x, None, freq, positions=pos, norm=True)
    assert none is None and torch.equal(got, want[0])
    spread = pos[:1].expand(6)  # strides of 0
    want, _ = pkg.rotary(x, None, freq, positions=spread.contiguous())
    q, k = x.clone(), x.clone()
    out = pkg.rotary(q, k, freq, positions=spread, out=(q, k))
    assert out[0] is q and torch.equal(q, want) and torch.equal(k, want)
    back = pkg.rotary_backward(q, k, freq, q, k, positions=spread, out=(q, k))
    assert back[2] is None and torch.allclose(q, x, atol=1e-5)


def test_rotary_frequencies():
    f = pkg.rotary_frequencies(64, base=500.0, device="cpu").numpy()
    assert np.allclose(f, 500.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-15)
    assert np.allclose(pkg.rotary_frequencies(64, base=500.0, factor=4.0, device="cpu").numpy(), f / 4, rtol=1e-15)
    g = pkg.rotary_frequencies(64, base=500.0, factor=4.0, original_length=256, device="cpu").numpy()
    turns = 256 * f / (2 * np.pi)
    assert np.array_equal(g[turns >= 4], f[turns >= 4]) and np.allclose(g[turns <= 1], f[turns <= 1] / 4, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all((g[mid] < f[mid]) & (g[mid] > f[mid] / 4))


# ----------------------------------------------------------------- gated MLP
def mlp_case(rows, K, F, O, dtype, kind="silu", seed=0, strided=False, big=1.0):
    import torch
    rng = np.random.default_rng(seed + rows + 3 * K + F)
    x, dy = draw(rng, (rows, K), dtype, big), draw(rng, (rows, O), dtype)
    wg, wu = draw(rng, (F, K), dtype, K ** -0.5), draw(rng, (F, K), dtype, K ** -0.5)
    wd = draw(rng, (O, F), dtype, F ** -0.5)
    t = [dev(v, dtype) for v in (x, wg, wu, wd, dy)]
    if strided:
        wide = torch.full((rows, K + O + 3), float("nan"), dtype=t[0].dtype, device=DEV)
        wide[:, 1:1 + K] = t[0]
        wide[:, K + 2:K + 2 + O] = t[4]
        t[0], t[4] = wide[:, 1:1 + K], wide[:, K + 2:K + 2 + O]
    y0 = pkg.gated_mlp(*t[:4], activation=kind)
    y, kept = pkg.gated_mlp_train(*t[:4], activation=kind)
    held = kept.clone()
    got = pkg.gated_mlp_backward(t[4], *t[:4], kept, activation=kind)
    assert torch.equal(y0, y) and torch.equal(held, kept)
    x, wg, wu, wd, dy = (v.astype(np.float64) for v in (x, wg, wu, wd, dy))
    rough = U16 if dtype == "bf16" else 0.0
    # a sum of n products: its chain of n additions, the products of the parts left out (4 U32), and a margin
    chain = lambda n: (n + 40) * U32  # noqa: E731
    ab = [np.abs(v) for v in (x, wg, wu, wd, dy)]
    g, u = x @ wg.T, x @ wu.T
    a, slope = ref.activation(g, kind)
    eg, eu = chain(K) * ab[0] @ ab[1].T, chain(K) * ab[0] @ ab[2].T
    # the activations' slopes are below 1.2 and their second derivatives below 1
    gate = (24 + 4 * np.abs(g)) * U32
    h = a * u
    eh = 1.2 * eg * np.abs(u) + np.abs(a) * eu + gate * np.abs(h) + gate * np.abs(u) * U32 + rough * np.abs(h)
    want = h @ wd.T
    close(y, want, eh @ ab[3].T + chain(F) * np.abs(h) @ ab[3].T + rough * np.abs(want) + 1e-30, "y")
    dh, edh = dy @ wd, chain(O) * ab[4] @ ab[3]
    eg, eu = eg + rough * np.abs(g), eu + rough * np.abs(u)
    dg, du = dh * u * slope, dh * a
    edg = (np.abs(u * slope) * edh + np.abs(dh * slope) * eu + np.abs(dh * u) * (eg + gate) + rough * np.abs(dg))
    edu = np.abs(a) * edh + np.abs(dh) * (1.2 * eg + gate * np.abs(a)) + rough * np.abs(du)
    rdx, rdg, rdu, rdd = ref.gated_mlp_backward(x, wg, wu, wd, dy, kind)
    adg, adu = np.abs(dg), np.abs(du)
    tols = ((edg + chain(2 * F) * adg) @ ab[1] + (edu + chain(2 * F) * adu) @ ab[2],
            (edg + chain(rows) * adg).T @ ab[0], (edu + chain(rows) * adu).T @ ab[0],
            ab[4].T @ (eh + chain(rows) * np.abs(h)))
    for v, w, tol, what in zip(got, (rdx, rdg, rdu, rdd), tols, ("dx", "dw_gate", "dw_up", "dw_down")):
        close(v, w, 1.01 * tol + rough * np.abs(w) + 1e-30, what)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,K,F,O", [(1, 1, 1, 1), (1, 64, 64, 64), (3, 8, 24, 16), (5, 17, 33, 9), (33, 100, 70, 50),
                                        (64, 256, 136, 72), (130, 72, 200, 130), (257, 130, 514, 65),
                                        (600, 64, 1000, 520), (1025, 72, 264, 257)])
def test_mlp(rows, K, F, O, dtype):
    mlp_case(rows, K, F, O, dtype)


@pytest.mark.parametrize("kind", ["silu", "gelu", "sigmoid"])
def test_mlp_activations(kind):
    for dtype in ("f32", "bf16"):
        mlp_case(70, 40, 56, 48, dtype, kind, big=3.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mlp_strided(dtype):
    mlp_case(70, 64, 72, 40, dtype, strided=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mlp_large_tiles(dtype):
    """Enough rows and columns for the largest tiles in every product, edges that end inside them."""
    mlp_case(4100, 264, 1800, 520, dtype)


def _mlp_check(x, wg, wu, wd, dy, dtype, kind="silu"):
    """mlp_case's comparison on the device, for sizes that take the host too long."""
    import torch
    y, kept = pkg.gated_mlp_train(x, wg, wu, wd, activation=kind)
    got = (y, *pkg.gated_mlp_backward(dy, x, wg, wu, wd, kept, activation=kind))
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    ab = [t.abs() for t in (x, wg, wu, wd, dy)]
    rows, K = x.shape
    F, O = wd.shape[1], wd.shape[0]
    rough = U16 if dtype == "bf16" else 0.0
    chain = lambda n: (n + 40) * U32  # noqa: E731
    g, u = x @ wg.T, x @ wu.T
    p = torch.sigmoid(g)
    a, slope = g * p, p + g * p * (1 - p)
    eg, eu = chain(K) * (ab[0] @ ab[1].T), chain(K) * (ab[0] @ ab[2].T)
    gate = (24 + 4 * g.abs()) * U32
    h = a * u
    eh = 1.2 * eg * u.abs() + a.abs() * eu + 2 * gate * h.abs() + rough * h.abs()
    dh, edh = dy @ wd, chain(O) * (ab[4] @ ab[3])
    eg, eu = eg + rough * g.abs(), eu + rough * u.abs()
    dg, du = dh * u * slope, dh * a
    edg = (u * slope).abs() * edh + (dh * slope).abs() * eu + (dh * u).abs() * (eg + gate) + rough * dg.abs()
    edu = a.abs() * edh + dh.abs() * (1.2 * eg + gate * a.abs()) + rough * du.abs()
    adg, adu = dg.abs(), du.abs()
    want = (h @ wd.T, dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ h)
    tols = (eh @ ab[3].T + chain(F) * (h.abs() @ ab[3].T),
            (edg + chain(2 * F) * adg) @ ab[1] + (edu + chain(2 * F) * adu) @ ab[2],
            (edg + chain(rows) * adg).T @ ab[0], (edu + chain(rows) * adu).T @ ab[0],
            ab[4].T @ (eh + chain(rows) * h.abs()))
    for v, w, tol, what in zip(got, want, tols, ("y", "dx", "dw_gate", "dw_up", "dw_down")):
        bad = (v.double() - w).abs() > 1.01 * tol + rough * w.abs() + 1e-30
        assert v.shape == w.shape and torch.isfinite(v).all() and not bad.any(), (what, int(bad.sum()))
        # the bounds grow with every sum; a piece that is missing or doubled shows in the whole
        assert float((v.double() - w).norm()) < (5e-3 if rough else 5e-6) * float(w.norm()), what


@pytest.mark.parametrize("dtype,odd", [("f32", True), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("rows,width,hidden", [
    (70, 40, 72), (2050, 2056, 72), (4100, 40, 2600), (8200, 1032, 136), (8200, 136, 4104), (2050, 2056, 1032),
    (2050, 264, 4104), (70, 2056, 4104), (12000, 136, 4104), (12000, 2056, 136), (8200, 2056, 1032),
    (2050, 2056, 2600), (12000, 2056, 264), (6000, 40, 72), (12000, 264, 136), (200, 1032, 2600), (8200, 2056, 4104)])
def test_mlp_every_tile(rows, width, hidden, dtype, odd):
    """Each product in each tile, whole, split along the contraction, and some tiles whole and some split: whatever the
    launch rule chooses between 70 and 12000 rows."""
    import torch
    gen = torch.Generator(device=DEV)
    gen.manual_seed(rows + hidden)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    K, F = (width - 5, hidden - 3) if odd else (width, hidden)
    put = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device=DEV) * std).to(dt)  # noqa: E731
    _mlp_check(put(rows, K), put(F, K, std=K ** -0.5), put(F, K, std=K ** -0.5), put(K, F, std=F ** -0.5),
               put(rows, K), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mlp_some_gradients(dtype):
    """Any of the gradients alone through the C interface (where the split of their sums may be another one)."""
    import itertools
    import torch
    from layer_lstm_forward_amd import block_ops as ops
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    put = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(dt)  # noqa: E731
    x, wg, wu, wd, dy = put(300, 72), put(200, 72), put(200, 72), put(64, 200), put(300, 64)
    _, kept = pkg.gated_mlp_train(x, wg, wu, wd)
    want = pkg.gated_mlp_backward(dy, x, wg, wu, wd, kept)
    shape = ops._pack_mlp(1 if dtype == "bf16" else 0, 0, 300, 72, 200, 64)
    n = ops.lstm_gated_mlp_backward_workspace_size(shape)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    for wanted in itertools.product((0, 1), repeat=4):
        out = [torch.full_like(t, float("nan")) if k else None for t, k in zip(want, wanted)]
        rc = ops.lstm_gated_mlp_backward(shape, x.data_ptr(), 72, wg.data_ptr(), wu.data_ptr(), wd.data_ptr(),
                                         kept.data_ptr(), kept.numel(), dy.data_ptr(), 64,
                                         *(None if t is None else t.data_ptr() for t in out), ws.data_ptr(), n,
                                         torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        for a, b in zip(out, want):
            assert a is None or torch.allclose(a.float(), b.float(), rtol=2 ** -6 if dtype == "bf16" else 1e-4,
                                               atol=1e-2 if dtype == "bf16" else 1e-4)


@pytest.mark.parametrize("rows", [9, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mlp_not_finite_rows_stay_alone(rows, dtype):
    import torch
    gen = torch.Generator(device=DEV)
    gen.manual_seed(8)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    put = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(dt)  # noqa: E731
    x, wg, wu, wd, dy = put(rows, 40), put(50, 40), put(50, 40), put(24, 50), put(rows, 24)
    y, kept = pkg.gated_mlp_train(x, wg, wu, wd)
    dx = pkg.gated_mlp_backward(dy, x, wg, wu, wd, kept)[0]
    keep = torch.arange(rows, device=DEV) != rows // 2
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[rows // 2, 3] = bad
        got, held = pkg.gated_mlp_train(z, wg, wu, wd)
        assert torch.equal(got[keep], y[keep]) and not torch.isfinite(got[~keep]).all()
        d = dy.clone()
        d[rows // 2, 3] = bad
        got = pkg.gated_mlp_backward(d, x, wg, wu, wd, kept)[0]
        assert torch.equal(got[keep], dx[keep]) and not torch.isfinite(got[~keep]).all()


@pytest.mark.parametrize("kind", ["silu", "gelu", "sigmoid"])
def test_mlp_large_values(kind):
    """Activations at their ends: no product of 0 and infinity."""
    for dtype in ("f32", "bf16"):
        for rows in (9, 90):
            mlp_case(rows, 24, 40, 16, dtype, kind, big=1e4)


def test_mlp_no_rows():
    import torch
    w = [torch.ones(s, device=DEV) for s in ((6, 4), (6, 4), (5, 6))]
    x = torch.empty(0, 4, device=DEV)
    y, kept = pkg.gated_mlp_train(x, *w)
    assert y.shape == (0, 5)
    dx, *dws = pkg.gated_mlp_backward(y, x, *w, kept)
    assert dx.shape == (0, 4)
    for d, v in zip(dws, w):
        assert d.shape == v.shape and not d.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mlp_no_rows_and_some_gradients(dtype):
    """Without rows a workspace may have no bytes; gradients that are not wanted stay out all the same."""
    import itertools
    import torch
    from layer_lstm_forward_amd import block_ops as ops
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    w = [torch.ones(64, 64, dtype=dt, device=DEV) for _ in range(3)]
    shape = ops._pack_mlp(1 if dtype == "bf16" else 0, 0, 0, 64, 64, 64)
    n = ops.lstm_gated_mlp_backward_workspace_size(shape)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    assert (ws is None) == (dtype == "bf16") and ops.lstm_gated_mlp_reserve_size(shape) == 0
    for wanted in itertools.product((0, 1), repeat=3):
        out = [torch.full_like(t, 3.0) if k else None for t, k in zip(w, wanted)]
        print(dtype, wanted, flush=True)
        rc = ops.lstm_gated_mlp_backward(shape, None, 64, *(t.data_ptr() for t in w), None, 0, None, 64, None,
                                         *(None if t is None else t.data_ptr() for t in out),
                                         None if ws is None else ws.data_ptr(), n,
                                         torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == 0 and all(t is None or not t.any() for t in out)


# ------------------------------------------------------- streams and graphs
def _fresh(dtype):
    import torch
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    put = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(dt)  # noqa: E731
    return dict(x=put(900, 2, 40), f=put(900, 2, 40), i=put(900, 2, 40), few=put(6, 40), pool=put(6, 40).float(),
                q=put(30, 2, 5, 24), k=put(30, 2, 3, 24), w=put(24), rows=put(300, 72), wg=put(200, 72),
                wu=put(200, 72), wd=put(72, 200), freq=pkg.rotary_frequencies(24, device=DEV))


def _everything(a):
    y, last = pkg.gated_recurrence(a["x"], a["f"], a["i"])
    out = [y, last, *pkg.gated_recurrence_backward(a["x"], a["f"], y, a["x"], a["i"])[:3]]
    short = [a[n][:50] for n in ("x", "f")]
    y, last = pkg.gated_recurrence(*short)
    out += [y, last, *pkg.gated_recurrence_backward(*short, y, short[0])[:2]]
    out += [pkg.gated_recurrence_step(a["few"], a["few"], a["pool"]), a["pool"]]
    more = dict(norm=True, q_weight=a["w"])
    q, k = pkg.rotary(a["q"], a["k"], a["freq"], **more)
    out += [q, k, *pkg.rotary_backward(a["q"], a["k"], a["freq"], q, k, **more)]
    weights = (a["wg"], a["wu"], a["wd"])
    for n in (7, 300):
        y, kept = pkg.gated_mlp_train(a["rows"][:n], *weights)
        out += [y, *pkg.gated_mlp_backward(y, a["rows"][:n], *weights, kept)]
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_another_stream(dtype):
    import torch
    a = _fresh(dtype)
    pool = a["pool"].clone()
    want = [t.clone() for t in _everything(a)]
    a["pool"].copy_(pool)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _everything(a)
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


def test_two_long_recurrences_at_once():
    """Two chains of tiles on two streams: each waits for tiles of its own alone."""
    import torch
    gen = torch.Generator(device=DEV)
    gen.manual_seed(8)
    x, f = (torch.randn(6000, 1, 1000, generator=gen, device=DEV).bfloat16() for _ in range(2))
    turned = x.flip(2).contiguous()
    want = [pkg.gated_recurrence(a, f) for a in (x, turned)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for k, a in enumerate((x, turned)):
            got[k].append(pkg.gated_recurrence(a, f, stream=sides[k].cuda_stream))
    torch.cuda.synchronize()
    for k in range(2):
        for y, last in got[k]:
            assert torch.equal(y, want[k][0]) and torch.equal(last, want[k][1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graph_replays(dtype):
    """Two graphs, replayed in turn with eager calls between, and their inputs changed."""
    import torch
    a = _fresh(dtype)
    pool, x = a["pool"].clone(), a["rows"].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _everything(a)
    side.synchronize()
    graphs = []
    for _ in range(2):
        a["pool"].copy_(pool)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = _everything(a)
        graphs.append((g, got))
    for turn in range(6):
        g, got = graphs[turn % 2]
        a["rows"].copy_(x * (1 + turn))
        a["pool"].copy_(pool)
        want = [t.clone() for t in _everything(a)]
        a["pool"].copy_(pool)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for y, z in zip(want, got):
            assert torch.equal(y, z)
        (torch.randn(1000, device=DEV) @ torch.randn(1000, device=DEV)).item()


# -------------------------------------------------- offsets that pass 32 bits
FAR = 2 ** 31 + 24  # elements from one batch row to the next


def _far(t):
    """t [T, 2, ...] with its batch rows FAR elements apart."""
    import torch
    row = t[:, 0].numel()
    flat = torch.empty(FAR + row, dtype=t.dtype, device=DEV)
    inner = t[:, 0].contiguous().stride()
    out = flat.as_strided(t.shape, (inner[0], FAR) + inner[1:])
    out.copy_(t)
    return out


@pytest.mark.parametrize("T", [40, 1500])
def test_recurrence_past_32_bits(T):
    import torch
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    x, f, dy = (torch.randn(T, 2, 24, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(3))
    y, last = pkg.gated_recurrence(x, f)
    want = [y, *pkg.gated_recurrence_backward(x, f, y, dy)[:2]]
    fx, ff, fy, fdy, fdx, fdf = (_far(t) for t in (x, f, torch.zeros_like(x), dy, torch.zeros_like(x),
                                                   torch.zeros_like(x)))
    _, far_last = pkg.gated_recurrence(fx, ff, out=(fy, torch.empty_like(last)))
    pkg.gated_recurrence_backward(fx, ff, fy, fdy, out=(fdx, fdf, None))
    for a, b in zip(want + [last], (fy, fdx, fdf, far_last)):
        assert torch.equal(a, b)


def test_recurrence_step_pool_past_32_bits():
    import torch
    n, W = 2 ** 20 + 5, 2052  # 2^31 + floats: 8.6 GB
    pool = torch.zeros(n, W, device=DEV)
    x = torch.randn(3, W, device=DEV)
    slots = torch.tensor([n - 1, 0, n - 2], dtype=torch.int32, device=DEV)
    state = torch.randn(3, W, device=DEV)
    pool[slots.long()] = state
    y = pkg.gated_recurrence_step(x, x, pool, slots=slots)
    assert torch.equal(y, pkg.gated_recurrence_step(x, x, state)) and torch.equal(pool[slots.long()], state)
    assert not pool[1:-2].any()


def test_rotary_past_32_bits():
    import torch
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    q, d = (torch.randn(6, 2, 3, 32, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    freq = pkg.rotary_frequencies(32, device=DEV)
    want, _ = pkg.rotary(q, None, freq, norm=True)
    wd, _, ww, _ = pkg.rotary_backward(q, None, freq, d, None, norm=True)
    fq, fo, fd, fdq = _far(q), _far(torch.zeros_like(q)), _far(d), _far(torch.zeros_like(q))
    pkg.rotary(fq, None, freq, norm=True, out=(fo, None))
    _, _, gw, _ = pkg.rotary_backward(fq, None, freq, fd, None, norm=True, out=(fdq, None))
    assert torch.equal(want, fo) and torch.equal(wd, fdq) and torch.equal(ww, gw)


def test_mlp_past_32_bits():
    """Hidden values past 2^32 elements: chosen rows and hidden units against fp64."""
    import torch
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    rows, K, F = 2 ** 19 + 5, 16, 8200
    put = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device=DEV) * std).to(torch.bfloat16)  # noqa: E731
    x, dy = put(rows, K), put(rows, K)
    wg, wu, wd = put(F, K, std=0.25), put(F, K, std=0.25), put(K, F, std=F ** -0.5)
    y, kept = pkg.gated_mlp_train(x, wg, wu, wd)
    dx, dg, du, dd = pkg.gated_mlp_backward(dy, x, wg, wu, wd, kept)

    def near(got, want):  # each rounding to 8 bits is off by 2^-9 rms at most; up to four of them
        assert float((got.double() - want).norm()) < 2 ** -7 * float(want.norm())

    def parts(x, dy, wg, wu, wd):
        x, dy, wg, wu, wd = (t.double() for t in (x, dy, wg, wu, wd))
        g, u = x @ wg.T, x @ wu.T
        p = torch.sigmoid(g)
        dh = dy @ wd
        return g * p * u, dh * u * (p + g * p * (1 - p)), dh * g * p

    for at in (slice(0, 3), slice(rows - 5, rows)):
        h, a, b = parts(x[at], dy[at], wg, wu, wd)
        near(y[at], h @ wd.double().T)
        near(dx[at], a @ wg.double() + b @ wu.double())
    at = slice(F - 4, F)
    h, a, b = parts(x, dy, wg[at], wu[at], wd[:, at])
    near(dg[at], a.T @ x.double())
    near(du[at], b.T @ x.double())
    near(dd[:, at], dy.double().T @ h)


# ------------------------------------------------------------------ together
class Block:
    """norm -> q, k, v -> rotary -> linear attention -> norm -> gated recurrence -> norm -> gated MLP, each with its
    residual sum, as a model has them; the same in fp64 for its differences."""

    W, H, D, HIDDEN, T, B = 48, 2, 24, 72, 21, 3

    def __init__(self):
        rng = np.random.default_rng(8)
        W, n = self.W, {}
        for name, shape in (("g1", (W,)), ("qkv", (W, 3 * W)), ("nq", (self.D,)), ("nk", (self.D,)), ("mix", (W, W)),
                            ("g2", (W,)), ("rec", (W, 3 * W)), ("g3", (W,)), ("wg", (self.HIDDEN, W)),
                            ("wu", (self.HIDDEN, W)), ("wd", (W, self.HIDDEN))):
            scale = shape[-1 if name.startswith("w") else 0] ** -0.5
            n[name] = 1 + 0.1 * rng.standard_normal(shape) if len(shape) == 1 else scale * rng.standard_normal(shape)
        n["x"] = rng.standard_normal((self.T, self.B, W))
        self.p = {k: v.astype(np.float32) for k, v in n.items()}
        self.decay = np.log(np.array([0.9, 0.99], np.float32))
        self.start = np.array([0, 100, 7], np.int32)
        self.dy = rng.standard_normal((self.T, self.B, W)).astype(np.float32)
        self.freq = pkg.rotary_frequencies(self.D, device="cpu").numpy()

    def exact(self, p):
        from oracle import ops as base
        T, B, W, H, D = self.T, self.B, self.W, self.H, self.D
        norm = lambda z, g: base.layer_norm(z.reshape(-1, W), g)[0].reshape(T, B, W)  # noqa: E731
        first = lambda t: t.transpose(1, 0, *range(2, t.ndim))  # noqa: E731
        q, k, v = (norm(p["x"], p["g1"]) @ p["qkv"]).reshape(T, B, 3, H, D).transpose(2, 0, 1, 3, 4)
        pos = np.arange(T)[:, None] + self.start
        q = ref.rotary(q, pos, self.freq, p["nq"], norm=True)
        k = ref.rotary(k, pos, self.freq, p["nk"], norm=True)
        o, _ = base.linear_attention(first(q), first(k), first(v), self.decay, D ** -0.5)
        z1 = p["x"] + first(o).reshape(T, B, W) @ p["mix"]
        parts = np.split(norm(z1, p["g2"]) @ p["rec"], 3, -1)
        z2 = z1 + first(ref.gated_recurrence(*(first(t) for t in parts))[0])
        m = ref.gated_mlp(norm(z2, p["g3"]).reshape(-1, W), p["wg"], p["wu"], p["wd"], "silu")
        return z2 + m.reshape(T, B, W)

    def forward(self, p):
        import torch
        T, B, W, H, D, t = self.T, self.B, self.W, self.H, self.D, {}
        t["n1"], t["m1"], t["r1"], _ = pkg.layer_norm(p["x"], p["g1"])
        wide = (t["n1"].view(-1, W) @ p["qkv"]).view(T, B, 3, H, D)
        t["q0"], t["k0"], t["v"] = wide.unbind(2)
        t["rot"] = dict(positions=torch.arange(T, dtype=torch.int32, device=DEV)[:, None] + dev(self.start),
                        q_weight=p["nq"], k_weight=p["nk"], norm=True)
        t["freq"] = dev(self.freq)
        t["q"], t["k"] = pkg.rotary(t["q0"], t["k0"], t["freq"], **t["rot"])
        t["o"], _ = pkg.linear_attention(t["q"], t["k"], t["v"], dev(self.decay))
        mixed = (t["o"].reshape(-1, W) @ p["mix"]).view(T, B, W)
        t["n2"], t["m2"], t["r2"], t["z1"] = pkg.layer_norm(mixed, p["g2"], residual=p["x"])
        t["xr"], t["f"], t["i"] = (t["n2"].view(-1, W) @ p["rec"]).view(T, B, 3 * W).split(W, -1)
        t["rec"], _ = pkg.gated_recurrence(t["xr"], t["f"], t["i"])
        t["n3"], t["m3"], t["r3"], t["z2"] = pkg.layer_norm(t["rec"], p["g3"], residual=t["z1"])
        m, t["kept"] = pkg.gated_mlp_train(t["n3"], p["wg"], p["wu"], p["wd"])
        return t["z2"] + m, t

    def backward(self, p, t, dy):
        import torch
        T, B, W, H, D, g = self.T, self.B, self.W, self.H, self.D, {}
        dn3, g["wg"], g["wu"], g["wd"] = pkg.gated_mlp_backward(dy, t["n3"], p["wg"], p["wu"], p["wd"], t["kept"])
        dz2, g["g3"], _ = pkg.layer_norm_backward(dn3, t["z2"], t["m3"], t["r3"], p["g3"], dsum=dy)
        wide = torch.empty(T, B, 3 * W, device=DEV)
        pkg.gated_recurrence_backward(t["xr"], t["f"], t["rec"], dz2, t["i"], out=wide.split(W, -1))
        wide = wide.view(-1, 3 * W)
        g["rec"] = t["n2"].view(-1, W).T @ wide
        dz1, g["g2"], _ = pkg.layer_norm_backward((wide @ p["rec"].T).view(T, B, W), t["z1"], t["m2"], t["r2"],
                                                  p["g2"], dsum=dz2)
        flat = dz1.view(-1, W)
        g["mix"] = t["o"].reshape(-1, W).T @ flat
        do = (flat @ p["mix"].T).view(T, B, H, D)
        wide = torch.empty(T, B, 3, H, D, device=DEV)
        dq, dk, dv = wide.unbind(2)
        pkg.linear_attention_backward(t["q"], t["k"], t["v"], dev(self.decay), do, out=(dq, dk, dv))
        _, _, g["nq"], g["nk"] = pkg.rotary_backward(t["q0"], t["k0"], t["freq"], dq, dk, out=(dq, dk), **t["rot"])
        wide = wide.view(-1, 3 * W)
        g["qkv"] = t["n1"].view(-1, W).T @ wide
        dx, g["g1"], _ = pkg.layer_norm_backward((wide @ p["qkv"].T).view(T, B, W), p["x"], t["m1"], t["r1"], p["g1"],
                                                 dsum=dz1)
        g["x"] = dx
        return g


def test_block_forward_and_gradients():
    b = Block()
    p64 = {n: v.astype(np.float64) for n, v in b.p.items()}
    p = {n: dev(v) for n, v in b.p.items()}
    want = b.exact(p64)
    y, t = b.forward(p)
    # fp32 throughout: chains of sums of at most 144 values of size one, norms in between
    assert np.max(np.abs(host(y) - want)) < 2000 * U32 * np.max(np.abs(want))
    grads = b.backward(p, t, dev(b.dy))
    rng = np.random.default_rng(9)
    for name, value in p64.items():
        u = rng.standard_normal(value.shape)
        h = 1e-5
        slope = ((b.exact({**p64, name: value + h * u}) - b.exact({**p64, name: value - h * u})) * b.dy).sum() / (2 * h)
        got = float((host(grads[name]) * u).sum())
        # differences: h^2 of a third derivative; gradients: sums of n products in fp32, each off by some hundred U32
        size = float(np.sqrt((host(grads[name]) ** 2).sum() * (u ** 2).mean()))
        assert abs(got - slope) < 1e-5 * abs(slope) + 4000 * U32 * size + 1e-6, (name, got, slope)


def test_block_token_by_token():
    """Serving: the same block on single tokens with states carried along."""
    import torch
    b = Block()
    p = {n: dev(v) for n, v in b.p.items()}
    want, _ = b.forward(p)
    B, W, H, D = b.B, b.W, b.H, b.D
    state, memory = torch.zeros(B, H, D, D, device=DEV), torch.zeros(B, W, device=DEV)
    freq, decay = dev(b.freq), dev(b.decay)
    for i in range(b.T):
        x = p["x"][i]
        n1 = pkg.layer_norm(x, p["g1"])[0]
        q, k, v = (n1 @ p["qkv"]).view(B, 3, H, D).unbind(1)
        q, k = pkg.rotary(q, k, freq, positions=dev(b.start + i), q_weight=p["nq"], k_weight=p["nk"], norm=True)
        o = pkg.linear_attention_step(q, k, v, decay, state)
        n2, _, _, z1 = pkg.layer_norm(o.view(B, W) @ p["mix"], p["g2"], residual=x)
        xr, f, g = (n2 @ p["rec"]).split(W, -1)
        r = pkg.gated_recurrence_step(xr, f, memory, input_gate=g)
        n3, _, _, z2 = pkg.layer_norm(r, p["g3"], residual=z1)
        y = z2 + pkg.gated_mlp(n3, p["wg"], p["wu"], p["wd"])
        assert float((y - want[i]).abs().max()) < 2000 * U32 * float(want.abs().max())
