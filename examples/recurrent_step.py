"""A small recurrent language model trained on a corpus and decoded from, on the library's operators.

Two blocks of gated recurrence: the embedding's rows come from det.embedding, layer norms from
det.layer_norm with the residual stream inside, each block's mixing over time from det.gated_scan, and
the loss from det.linear_cross_entropy, which never stores a logit.  Every sum in these operators and in
their gradients has a fixed order, so a step's loss and gradients do not move from run to run on
their account (the matrix products between them are torch's).  Decoding keeps one float32 state a block
and steps it in place, a token at a time.

    python examples/recurrent_step.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from scan_fixed_order_amd import det  # noqa: E402

VOCAB, WIDTH, BLOCKS = 1000, 128, 2


class Recurrent:
    def __init__(self, device, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, scale=1.0):
            w = torch.randn(shape, generator=g) * scale / shape[-1] ** 0.5
            return w.to(device).requires_grad_(True)

        def ones():
            return torch.ones(WIDTH, device=device, requires_grad=True)

        def zeros():
            return torch.zeros(WIDTH, device=device, requires_grad=True)

        self.embed, self.out = weight(VOCAB, WIDTH), weight(VOCAB, WIDTH)
        self.blocks = [{"gate": weight(WIDTH, WIDTH), "x": weight(WIDTH, WIDTH),
                        "mix": weight(WIDTH, WIDTH, scale=0.5), "norm": ones(), "shift": zeros()}
                       for _ in range(BLOCKS)]
        self.norm, self.shift = ones(), zeros()
        self.parameters = [self.embed, self.out, self.norm, self.shift] + [
            p for b in self.blocks for p in b.values()]

    def hidden(self, tokens, lengths):
        """[batch, t, width] behind the last norm, for tokens [batch, t] of which lengths count."""
        h = det.embedding(self.embed, tokens, WIDTH ** 0.5)
        out = None
        for b in self.blocks:
            if out is None:
                n = det.layer_norm(h, b["norm"], b["shift"])
            else:
                n, h = det.layer_norm(out, b["norm"], b["shift"], residual=h)
            s, _ = det.gated_scan(n @ b["gate"], n @ b["x"], sigmoid=True, lengths=lengths)
            out = s @ b["mix"]
        return det.layer_norm(out, self.norm, self.shift, residual=h)[0]


def step(model, tokens, lengths, lr=0.5):
    """One step of gradient descent on sequences [batch, t + 1], with numbers outside the vocabulary (such
    as -1) past their lengths; returns the loss."""
    x, targets = tokens[:, :-1].contiguous(), tokens[:, 1:].contiguous()
    loss = det.linear_cross_entropy(model.hidden(x, lengths), model.out, targets)
    loss = loss.sum() / ((targets >= 0) & (targets < VOCAB)).sum()
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
    batch = prompt.shape[0]
    states = [torch.zeros(batch, WIDTH, device=prompt.device) for _ in model.blocks]

    def walk(ids):
        h = det.det_embedding(model.embed, ids, WIDTH ** 0.5)
        out = None
        for b, state in zip(model.blocks, states):
            r = det.det_layer_norm(h if out is None else out, b["norm"], b["shift"],
                                   residual=None if out is None else h)
            h = r.h
            s = det.det_gated_scan(r.y @ b["gate"], r.y @ b["x"], state=state, sigmoid=True)
            state.copy_(s.state)
            out = s.h @ b["mix"]
        return det.det_layer_norm(out, model.norm, model.shift, residual=h).y[:, -1].contiguous()

    y, ids, logps = walk(prompt), [], []
    for _ in range(tokens):
        best = (y @ model.out.t()).argmax(-1)
        logps.append(-det.det_linear_cross_entropy(y, model.out, best).loss)
        ids.append(best)
        y = walk(best[:, None].contiguous())
    return torch.stack(ids, 1), torch.stack(logps, 1)


def corpus(device, batch=16, steps=96, seed=1):
    """Sequences that count upwards by a stride of their own; of different lengths, -1 past them."""
    g = torch.Generator().manual_seed(seed)
    start = torch.randint(0, VOCAB, (batch, 1), generator=g)
    stride = torch.randint(1, 4, (batch, 1), generator=g)
    tokens = (start + stride * torch.arange(steps + 1)) % VOCAB
    lengths = torch.randint(2, steps + 1, (batch,), generator=g)
    tokens = torch.where(torch.arange(steps + 1) <= lengths[:, None], tokens, -1)
    return tokens.to(device), lengths.to(torch.int32).to(device)


def run(steps=20, device="cuda", seed=0):
    model = Recurrent(device, seed)
    tokens, lengths = corpus(device)
    losses = [float(step(model, tokens, lengths)) for _ in range(steps)]
    return model, tokens, losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    steps = ap.parse_args().steps
    model, tokens, losses = run(steps)
    again = run(steps)[2]
    print("loss %.4f -> %.4f, a second run's losses %s" % (
        losses[0], losses[-1], "are the same" if again == losses else "differ"))
    ids, logps = decode(model, tokens[:, :2].contiguous(), 12)
    print("decoded", ids[0].tolist(), "at log probabilities", [round(v, 3) for v in logps[0].tolist()])


if __name__ == "__main__":
    main()
