"""A small recurrent sequence model trained and served with this library's kernels.

    embedding -> LSTM -> layer norm (+ residual) -> q, k, v -> linear attention with a decay for each head
              -> layer norm (+ residual) -> logits

The task is associative recall: a sequence of pairs (key, value) followed by a key, whose value the model has to
answer.  Training runs the LSTM's forward_train / backward, linear_attention / linear_attention_backward,
layer_norm / layer_norm_backward and adamw_step; the dense projections are plain torch products.  Afterwards a
sequence is answered once as a whole and once token by token (linear_attention_step on the carried state), and the two
have to agree.

    python examples/train_sequence_model.py [--steps 800] [--state-bits 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import layer_lstm_forward_amd as lib  # noqa: E402

SYMBOLS, PAIRS, WIDTH, HEADS, DIM = 32, 12, 128, 4, 32
SEQ = 2 * PAIRS + 1


def batch(rows, gen, device):
    """tokens [SEQ, rows]: key, value, key, value, ..., key; the answer to the last key."""
    keys = torch.rand(rows, SYMBOLS, generator=gen, device=device).argsort(1)[:, :PAIRS]
    values = torch.randint(SYMBOLS, (rows, PAIRS), generator=gen, device=device)
    asked = torch.randint(PAIRS, (rows, 1), generator=gen, device=device)
    pairs = torch.stack([keys, values + SYMBOLS], 2).reshape(rows, 2 * PAIRS)
    return torch.cat([pairs, keys.gather(1, asked)], 1).T.contiguous(), values.gather(1, asked)[:, 0]


class Model:
    def __init__(self, device, gen):
        def draw(*shape, scale):
            return torch.randn(*shape, generator=gen, device=device) * scale

        self.lstm = lib.LSTM(WIDTH, WIDTH, dtype="f32")
        k = WIDTH ** -0.5
        self.p = {
            "embed": draw(2 * SYMBOLS, WIDTH, scale=1.0),
            "w_ih": draw(4 * WIDTH, WIDTH, scale=k), "w_hh": draw(4 * WIDTH, WIDTH, scale=k),
            "b_ih": torch.zeros(4 * WIDTH, device=device), "b_hh": torch.zeros(4 * WIDTH, device=device),
            "g1": torch.ones(WIDTH, device=device), "c1": torch.zeros(WIDTH, device=device),
            "qkv": draw(WIDTH, 3 * HEADS * DIM, scale=k), "mix": draw(HEADS * DIM, WIDTH, scale=k),
            "g2": torch.ones(WIDTH, device=device), "c2": torch.zeros(WIDTH, device=device),
            "out": draw(WIDTH, SYMBOLS, scale=k),
        }
        # heads that forget within the sequence and heads that keep all of it
        self.decay = torch.log(torch.tensor([0.9, 0.97, 0.99, 1.0], device=device))

    def lstm_weights(self):
        return [self.p[n] for n in ("w_ih", "w_hh", "b_ih", "b_hh")]

    def forward(self, tokens):
        p, t = self.p, {}
        T, B = tokens.shape
        t["x"] = p["embed"][tokens]
        t["h"], _, _, t["reserve"] = self.lstm.forward_train(t["x"], self.lstm_weights())
        t["n1"], t["m1"], t["r1"], t["z1"] = lib.layer_norm(t["h"], p["g1"], p["c1"], residual=t["x"])
        wide = (t["n1"].view(T * B, WIDTH) @ p["qkv"]).view(T, B, 3, HEADS, DIM)
        t["q"], t["k"], t["v"] = wide.unbind(2)  # strided views: the operator reads them in place
        t["o"], t["state"] = lib.linear_attention(t["q"], t["k"], t["v"], self.decay)
        mixed = (t["o"].view(T * B, HEADS * DIM) @ p["mix"]).view(T, B, WIDTH)
        t["n2"], t["m2"], t["r2"], t["z2"] = lib.layer_norm(mixed, p["g2"], p["c2"], residual=t["z1"])
        return t["n2"][-1] @ p["out"], t

    def backward(self, tokens, t, dlogits):
        """Gradients of every parameter, in the order of self.p."""
        p, g = self.p, {}
        T, B = tokens.shape
        g["out"] = t["n2"][-1].T @ dlogits
        dn2 = torch.zeros_like(t["n2"])
        dn2[-1] = dlogits @ p["out"].T
        dz2, g["g2"], g["c2"] = lib.layer_norm_backward(dn2, t["z2"], t["m2"], t["r2"], p["g2"])
        flat = dz2.view(T * B, WIDTH)
        g["mix"] = t["o"].view(T * B, HEADS * DIM).T @ flat
        do = (flat @ p["mix"].T).view(T, B, HEADS, DIM)
        dwide = torch.empty(T, B, 3, HEADS, DIM, device=tokens.device)
        lib.linear_attention_backward(t["q"], t["k"], t["v"], self.decay, do, out=dwide.unbind(2))
        dwide = dwide.view(T * B, 3 * HEADS * DIM)
        g["qkv"] = t["n1"].view(T * B, WIDTH).T @ dwide
        dn1 = (dwide @ p["qkv"].T).view(T, B, WIDTH)
        # dz2 is also the gradient of the residual stream z1
        dz1, g["g1"], g["c1"] = lib.layer_norm_backward(dn1, t["z1"], t["m1"], t["r1"], p["g1"], dsum=dz2)
        dx, _, _, dw = self.lstm.backward(t["x"], self.lstm_weights(), t["h"], t["reserve"], dz1)
        g["w_ih"], g["w_hh"], g["b_ih"], g["b_hh"] = dw
        g["embed"] = torch.zeros_like(p["embed"]).index_add_(0, tokens.reshape(-1), (dx + dz1).view(T * B, WIDTH))
        return [g[n] for n in p]

    def answer_token_by_token(self, tokens):
        p = self.p
        T, B = tokens.shape
        state = torch.zeros(B, HEADS, DIM, DIM, device=tokens.device)
        h = c = torch.zeros(1, B, WIDTH, device=tokens.device)
        for i in range(T):
            x = p["embed"][tokens[i:i + 1]]
            y, h, c = self.lstm.forward(x, self.lstm_weights(), h, c)
            n1, _, _, z1 = lib.layer_norm(y[0], p["g1"], p["c1"], residual=x[0])
            q, k, v = (n1 @ p["qkv"]).view(B, 3, HEADS, DIM).unbind(1)
            o = lib.linear_attention_step(q, k, v, self.decay, state)
            n2, *_ = lib.layer_norm(o.view(B, HEADS * DIM) @ p["mix"], p["g2"], p["c2"], residual=z1)
        return n2 @ p["out"]


def train(steps=800, rows=128, state_bits=32, seed=0, device="cuda", report=print):
    """Returns (first loss, last loss, largest difference between the two ways to answer)."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    model = Model(torch.device(device, torch.cuda.current_device()), gen)
    params = list(model.p.values())
    m, v, scales = lib.adamw_states(params, bits=state_bits)
    decay = [0.01 if x.dim() > 1 else 0.0 for x in params]  # none on biases and norms
    first = last = None
    for step in range(1, steps + 1):
        tokens, answer = batch(rows, gen, params[0].device)
        logits, kept = model.forward(tokens)
        chance = torch.log_softmax(logits, -1)
        loss = -chance.gather(1, answer[:, None]).mean()
        dlogits = chance.exp()
        dlogits[torch.arange(rows, device=answer.device), answer] -= 1
        grads = model.backward(tokens, kept, dlogits / rows)
        # clipping: the factor stays on the device
        norm = torch.sqrt(sum((g * g).sum() for g in grads))
        lib.adamw_step(params, grads, m, v, step=step, lr=3e-3 * min(1.0, step / 50), weight_decay=decay,
                       scales=scales, grad_scale=(1.0 / norm.clamp(min=1.0)).view(1), seed=step)
        if step == 1:
            first = float(loss)
        if step % 100 == 0 or step == steps:
            last = float(loss)
            report(f"step {step}: loss {last:.4f}")
    tokens, _ = batch(16, gen, params[0].device)
    apart = float((model.forward(tokens)[0] - model.answer_token_by_token(tokens)).abs().max())
    return first, last, apart


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=800)
    ap.add_argument("--rows", type=int, default=128)
    ap.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    a = ap.parse_args()
    before, after, off = train(a.steps, a.rows, a.state_bits)
    print(f"loss {before:.3f} -> {after:.3f}; whole sequence against token by token: {off:.2e}")
