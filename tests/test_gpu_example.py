"""The example model: its gradients against differences, that it learns with both kinds of optimizer state, and that
whole sequences and single tokens give one answer."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_sequence_model.py")


def _example():
    spec = importlib.util.spec_from_file_location("train_sequence_model", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("bits", [32, 8])
def test_example_learns(bits):
    ex = _example()
    first, last, apart = ex.train(state_bits=bits, report=lambda s: print(s, flush=True))
    # chance is log 32 = 3.47 at the start; below half of it the model answers from the sequence
    assert first > 3.0 and last < 0.5 * first, (first, last)
    # fp32 throughout: two orders of the same sums over 25 tokens
    assert apart < 1e-2, apart


def test_example_gradients_are_differences():
    """Along a random direction of all parameters: the loss's slope from the gradients and from the loss."""
    import torch
    ex = _example()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    model = ex.Model(torch.device("cuda", 0), gen)
    tokens, answer = ex.batch(32, gen, torch.device("cuda", 0))

    def loss():
        logits, kept = model.forward(tokens)
        chance = torch.log_softmax(logits.double(), -1)
        return float(-chance.gather(1, answer[:, None]).mean()), logits, kept

    _, logits, kept = loss()
    d = torch.softmax(logits, -1)
    d[torch.arange(32, device="cuda"), answer] -= 1
    grads = model.backward(tokens, kept, d / 32)
    for n, (name, p) in enumerate(model.p.items()):
        u = torch.randn(p.shape, generator=gen, device="cuda")
        u *= p.norm() / u.norm() if p.norm() > 0 else 1.0
        slope = float((grads[n].double() * u.double()).sum())
        h, keep = 1e-2, p.clone()
        p.copy_(keep + h * u)
        up = loss()[0]
        p.copy_(keep - h * u)
        down = loss()[0]
        p.copy_(keep)
        # the loss is about 3.5 in fp32 (2^-22 of it over 2h: 4e-5); third derivatives times h^2 / 6 at slopes of
        # about one: below 2e-3
        assert abs((up - down) / (2 * h) - slope) < 5e-3 + 0.02 * abs(slope), (name, (up - down) / (2 * h), slope)
