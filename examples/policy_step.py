"""A small decoder trained by policy gradient and sampled from, on the language-model operators.

One attention block with a learned relative position bias: the embedding's rows come from
det.gather, both norms from det.rms_norm, the attention's scores get their bias and masks from
det.relative_bias, and det.token_logprobs turns the logits into the log probabilities and entropies
that the loss is made of.  Every sum in these operators and in their gradients has a fixed order,
so a step's loss and gradients do not move from run to run on their account (the matrix products
are torch's).  Decoding calls the same operators for one token at a time, the last norm with an
8-bit output as an 8-bit projection would take it, and scores its samples with alternatives.

    python examples/policy_step.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from scan_fixed_order_amd import det  # noqa: E402

VOCAB, WIDTH, HEADS, BUCKETS, DISTANCE = 1000, 128, 4, 32, 128


class Policy:
    def __init__(self, device, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, scale=1.0):
            w = torch.randn(shape, generator=g) * scale / shape[0] ** 0.5
            return w.to(device).requires_grad_(True)

        self.embed = weight(VOCAB, WIDTH, scale=VOCAB ** 0.5)
        self.q, self.k, self.v, self.o = (weight(WIDTH, WIDTH) for _ in range(4))
        self.out = weight(WIDTH, VOCAB)
        self.bias = weight(BUCKETS, HEADS)
        self.norm1, self.norm2 = (torch.ones(WIDTH, device=device, requires_grad=True)
                                  for _ in range(2))
        self.parameters = [self.embed, self.q, self.k, self.v, self.o, self.out, self.bias,
                           self.norm1, self.norm2]

    def heads(self, x, w):
        b, t, _ = x.shape
        return (x @ w).view(b, t, HEADS, -1).transpose(1, 2).contiguous()

    def logits(self, tokens, lengths):
        """[batch, t, vocab] for tokens [batch, t] (int32), of which lengths count."""
        b, t = tokens.shape
        x = det.gather(self.embed, tokens.reshape(-1)).view(b, t, WIDTH)
        n = det.rms_norm(x, self.norm1)
        q, k, v = (self.heads(n, w) for w in (self.q, self.k, self.v))
        scores = q @ k.transpose(2, 3).contiguous() * (WIDTH // HEADS) ** -0.5
        scores = det.relative_bias(self.bias, t, t, scores, DISTANCE, bidirectional=False,
                                   causal=True, lengths=lengths)
        # a padded query sees no key: its row of -inf becomes a row of zeros
        p = torch.where(scores.amax(-1, keepdim=True) > -float("inf"), scores, 0.0).softmax(-1)
        a = (p @ v).transpose(1, 2).reshape(b, t, WIDTH) @ self.o
        y, _ = det.rms_norm(a, self.norm2, residual=x)
        return y @ self.out


def step(model, tokens, lengths, advantage, lr=0.2, entropy_bonus=1e-3):
    """One policy-gradient step on sampled tokens; returns the loss."""
    logits = model.logits(tokens[:, :-1].contiguous(), lengths)
    at = torch.arange(tokens.shape[1] - 1, device=tokens.device)
    # positions past a sequence's length are not scored
    targets = torch.where(at < lengths[:, None] - 1, tokens[:, 1:].long(), -100)
    logp, entropy = det.token_logprobs(logits, targets)
    entropy = torch.where(targets >= 0, entropy, 0.0)      # it is returned for every position
    scored = (targets >= 0).sum()
    loss = -((logp * advantage[:, None]).sum() + entropy_bonus * entropy.sum()) / scored
    for p in model.parameters:
        p.grad = None
    loss.backward()
    with torch.no_grad():
        for p in model.parameters:
            p -= lr * p.grad
    return loss.detach()


@torch.no_grad()
def decode(model, prompt, tokens):
    """Greedy continuation of prompt [batch, t] by `tokens` tokens; also their log probabilities."""
    b, t = prompt.shape
    prompt = prompt.long()
    x = model.embed[prompt]
    n = det.det_rms_norm(x, model.norm1).y
    keys, values = model.heads(n, model.k), model.heads(n, model.v)
    last, logps, ids = x[:, -1], [], []
    for i in range(tokens):
        n = det.det_rms_norm(last, model.norm1).y[:, None]
        if i:      # the prompt's own keys and values are there already
            keys = torch.cat([keys, model.heads(n, model.k)], 2)
            values = torch.cat([values, model.heads(n, model.v)], 2)
        length = keys.shape[2]
        scores = model.heads(n, model.q) @ keys.transpose(2, 3).contiguous() * (WIDTH // HEADS) ** -0.5
        scores = det.det_relative_bias(model.bias, 1, length, scores, DISTANCE, bidirectional=False,
                                       causal=True, q_offset=length - 1, out=scores)
        a = (scores.softmax(-1) @ values).transpose(1, 2).reshape(b, WIDTH) @ model.o
        r = det.det_rms_norm(a, model.norm2, residual=last, quant=torch.float8_e4m3fn, group=32)
        y = (r.y.float().view(b, -1, 32) * r.scales[..., None]).view(b, WIDTH)
        logits = y @ model.out
        best = det.det_token_logprobs(logits, torch.zeros(b, dtype=torch.long, device=x.device),
                                      top=5)
        token = best.top_ids[:, 0]
        logps.append(best.top_logp[:, 0])
        ids.append(token)
        last = model.embed[token]
    return torch.stack(ids, 1), torch.stack(logps, 1)


def run(steps=20, device="cuda", seed=0):
    model = Policy(device, seed)
    g = torch.Generator().manual_seed(seed + 1)
    tokens = torch.randint(0, VOCAB, (8, 65), generator=g, dtype=torch.int32).to(device)
    lengths = torch.tensor([65, 65, 40, 33, 65, 7, 2, 50], dtype=torch.int32, device=device)
    advantage = torch.ones(8, device=device)
    losses = [float(step(model, tokens, lengths, advantage)) for _ in range(steps)]
    return model, tokens, losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    steps = ap.parse_args().steps
    model, tokens, losses = run(steps)
    again = run(steps)[2]
    print("loss %.4f -> %.4f, a second run's losses %s" % (
        losses[0], losses[-1], "are the same" if again == losses else "differ"))
    ids, logps = decode(model, tokens[:, :16], 12)
    print("decoded", ids[0].tolist(), "at log probabilities", [round(v, 3) for v in logps[0].tolist()])


if __name__ == "__main__":
    main()
