"""Embedding, layer norm, gated recurrence and linear cross entropy together, as
examples/recurrent_step.py uses them."""
import importlib.util
import os

import pytest
import torch

from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "recurrent_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("recurrent_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_and_decoding_run(dev, example):
    model, tokens, losses = example.run(6)
    assert all(0 < v < 100 for v in losses)
    assert all(torch.isfinite(p).all() and torch.isfinite(p.grad).all() for p in model.parameters)
    ids, logps = example.decode(model, tokens[:, :2].contiguous(), 5)
    assert ids.shape == (16, 5) and (logps <= 1e-6).all() and torch.isfinite(logps).all()


def plain(example, p, tokens, lengths):
    """The model's loss and hidden rows by torch's operations in the parameters' type."""
    embed, out, norm, shift, *rest = p

    def layer(h, w, b):
        h = h - h.mean(-1, keepdim=True)
        return h * (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w + b

    x, targets = tokens[:, :-1], tokens[:, 1:]
    h = torch.where((x >= 0)[..., None], embed[x.clamp_min(0)], 0.0) * example.WIDTH ** 0.5
    add = None
    for i in range(example.BLOCKS):
        gate, inp, mix, w, b = rest[5 * i:5 * i + 5]
        h = h if add is None else h + add
        n = layer(h, w, b)
        a, u = torch.sigmoid(n @ gate), n @ inp
        s, hs = torch.zeros_like(h[:, 0]), []
        for t in range(x.shape[1]):
            live = (t < lengths)[:, None]
            s = torch.where(live, a[:, t] * s + (1 - a[:, t]) * u[:, t], s)
            hs.append(torch.where(live, s, 0.0))
        add = torch.stack(hs, 1) @ mix
    y = layer(h + add, norm, shift)
    log = (y @ out.t()).log_softmax(-1)
    picked = log.gather(-1, targets.clamp_min(0)[..., None])[..., 0]
    on = targets >= 0
    return -torch.where(on, picked, 0.0).sum() / on.sum(), y


def test_gradients_of_the_model_against_64_bits(dev, example):
    model = example.Recurrent(dev, 3)
    tokens, lengths = example.corpus(dev, batch=5, steps=37, seed=4)
    before = [v.detach().clone() for v in model.parameters]
    loss = example.step(model, tokens, lengths, lr=0.0)
    p = [v.double().requires_grad_(True) for v in before]
    want, _ = plain(example, p, tokens, lengths)
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 1e-5 * float(want.detach())
    for got, w in zip(model.parameters, p):
        # f32 products and sums of up to 1000 terms, through two blocks and 37 steps
        assert ((got.grad.double() - w.grad).abs() <= 5e-4 * w.grad.abs().max()).all()


def test_a_step_repeats_and_does_not_learn_from_padding(dev, example):
    tokens, lengths = example.corpus(dev)
    steps = []
    for t in (tokens, tokens, torch.where(tokens < 0, example.VOCAB + 7, tokens)):
        model = example.Recurrent(dev, 0)
        loss = example.step(model, t, lengths)
        steps.append((loss, [v.grad for v in model.parameters]))
    for loss, grads in steps[1:]:
        # past a length nothing is scored and no token is known, whatever number stands there
        assert torch.equal(loss, steps[0][0])
        for a, b in zip(grads, steps[0][1]):
            assert torch.equal(a, b)


def test_decoding_follows_the_sequence(dev, example):
    """Token by token from kept states, as the whole sequence at once: the same numbers but for the
    order in which spans are composed and torch's products over other shapes."""
    model = example.Recurrent(dev, 1)
    prompt = torch.randint(0, example.VOCAB, (3, 9), device=dev)
    ids, logps = example.decode(model, prompt, 6)
    whole = torch.cat([prompt, ids], 1)
    y = model.hidden(whole, torch.full((3,), 15, dtype=torch.int32, device=dev))
    loss = det.det_linear_cross_entropy(y[:, 8:14].contiguous(), model.out, ids).loss
    assert ((loss + logps).abs() <= 1e-4).all()
