"""The language-model operators together, as examples/policy_step.py uses them."""
import importlib.util
import os

import pytest
import torch

from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "policy_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("policy_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_lowers_the_loss_and_decoding_follows_it(dev, example):
    model, tokens, losses = example.run(12)
    assert all(l == l and abs(l) < 100 for l in losses) and losses[-1] < losses[0] - 0.5
    assert all(torch.isfinite(p).all() and torch.isfinite(p.grad).all() for p in model.parameters)
    ids, logps = example.decode(model, tokens[:, :9], 5)
    assert ids.shape == (8, 5) and (logps <= 0).all() and torch.isfinite(logps).all()


def test_gradients_of_the_block_against_64_bits(dev, example):
    """The block's gradients through the operators against torch's through the formulas."""
    model = example.Policy(dev, 3)
    tokens = torch.randint(0, example.VOCAB, (3, 21), device=dev, dtype=torch.int32)
    lengths = torch.tensor([20, 9, 1], dtype=torch.int32, device=dev)
    logits = model.logits(tokens[:, :-1].contiguous(), lengths)
    targets = torch.where(torch.arange(20, device=dev) < lengths[:, None], tokens[:, 1:].long(), -100)
    logp, entropy = det.token_logprobs(logits, targets)
    (logp.sum() + 0.1 * entropy.sum()).backward()

    p = [v.detach().double().requires_grad_(True) for v in model.parameters]
    embed, q, k, v, o, out, bias, n1, n2 = p
    x = embed[tokens[:, :-1].long()]

    def norm(h, w):
        return h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w

    def heads(n, w):
        return (n @ w).view(3, 20, example.HEADS, -1).transpose(1, 2)

    n = norm(x, n1)
    from lm_reference import bucket
    i, j = torch.arange(20)[:, None], torch.arange(20)[None]
    bk = torch.tensor([[bucket(int(b - a), 32, 128, False) for b in range(20)] for a in range(20)])
    scores = heads(n, q) @ heads(n, k).transpose(2, 3) * (example.WIDTH // example.HEADS) ** -0.5
    scores = scores + bias[bk.to(dev)].permute(2, 0, 1)
    at = lengths.cpu()[:, None, None]
    left = ((j <= i) & (j < at) & (i < at)).to(dev)[:, None]
    scores = torch.where(left, scores, -float("inf"))
    some = left.any(-1, keepdim=True)
    prob = torch.where(some, scores, 0.0).softmax(-1)
    a = (prob @ heads(n, v)).transpose(1, 2).reshape(3, 20, -1) @ o
    log = (norm(a + x, n2) @ out).log_softmax(-1)
    ok = targets >= 0
    picked = log.gather(-1, targets.clamp_min(0)[..., None])[..., 0]
    (torch.where(ok, picked, 0.0).sum() - 0.1 * (log.exp() * log).sum()).backward()
    for got, want in zip(model.parameters, p):
        # f32 products and sums of up to 1000 terms, through three layers
        size = want.grad.abs().max()
        assert ((got.grad.double() - want.grad).abs() <= 2e-4 * size).all()


def test_a_step_does_not_learn_from_padding(dev, example):
    """Loss and gradients are the same whatever stands past each length.  Of the embedding's
    gradient the zeros that padding adds may regroup a row's sum (at most 8 rows of one token here,
    3 levels of 2^-24 each, relative to 8 times the largest)."""
    g = torch.Generator().manual_seed(5)
    tokens, other = (torch.randint(0, example.VOCAB, (5, 33), generator=g, dtype=torch.int32).to(dev)
                     for _ in range(2))
    lengths = torch.tensor([33, 9, 2, 20, 1], dtype=torch.int32, device=dev)
    other = torch.where(torch.arange(33, device=dev) < lengths[:, None], tokens, other)
    steps = []
    for t in (tokens, other):
        model = example.Policy(dev, 0)
        loss = example.step(model, t, lengths, torch.ones(5, device=dev), entropy_bonus=0.5)
        steps.append((loss, [p.grad for p in model.parameters]))
    (loss, grads), (again, same) = steps
    assert not torch.equal(tokens, other) and torch.equal(loss, again)
    for a, b in zip(grads, same):
        assert ((a - b).abs() <= 8 * 3 * 2.0 ** -24 * a.abs().max()).all()
