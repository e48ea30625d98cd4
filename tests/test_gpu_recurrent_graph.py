"""Embedding, layer norm, gated recurrence and linear cross entropy captured into one graph and replayed
on changed inputs, with eager work between the replays: every replay has the bits of direct calls."""
import pytest
import torch

from lm_reference import randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16], ids=["f32", "f16", "bf16"])
def test_replays_match_direct_calls(dev, t):
    batch, steps, d, vocab = 2, 700, 96, 1500
    n = batch * steps
    table, w = randn((vocab, d), t, dev, 1), randn((d,), t, dev, 2)
    gate, dh = randn((batch, steps, d), t, dev, 3), randn((batch, steps, d), t, dev, 4)
    ids = torch.randint(0, vocab, (batch, steps), device=dev)
    many = torch.randint(0, vocab, (66000,), device=dev)      # through the radix sort
    rows = randn((66000, 8), t, dev, 5)
    lens = torch.tensor([700, 410], dtype=torch.int32, device=dev)
    state, kept = randn((batch, d), torch.float32, dev, 6), torch.zeros(batch, d, device=dev)
    dl = randn((batch, steps), torch.float32, dev, 7)

    def run():
        x = det.det_embedding(table, ids, 2.0)
        a = det.det_layer_norm(x, w, w, residual=gate)
        r = det.det_gated_scan(gate, a.y, state, True, lens)
        one = det.det_gated_scan(gate[:, :1].contiguous(), x[:, :1].contiguous(), kept, True, state_out=kept)
        loss = det.det_linear_cross_entropy(r.h, table, ids)
        dx, dw = det.det_linear_cross_entropy_backward(r.h, table, ids, loss.lse, dl)
        back = det.det_gated_scan_backward(dx, gate, a.y, r.h, state, state, True, lens)
        norm = det.det_layer_norm_backward(back[1], a.h, w, a.mean, a.rstd, dh)
        return [x, *a, *r, one.h, *loss, dx, dw, *back, *norm, det.det_embedding_backward(norm[0], ids, vocab),
                det.det_embedding_backward(rows, many, vocab)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    assert n == outs[0].shape[0] * outs[0].shape[1]
    for i in range(4):
        for k, v in enumerate((gate, dh, rows, table)):
            v.copy_(randn(v.shape, t, dev, 100 * i + k))
        ids.copy_(torch.randint(-1, vocab + 1, ids.shape, device=dev))
        lens.copy_(torch.tensor([700 - i, 3 + 50 * i], dtype=torch.int32))
        for o in outs:
            o.view(-1).view(torch.uint8).fill_(0xA5)
        kept.fill_(0.5)
        want = run()
        end = kept.clone()
        kept.fill_(0.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert same_bits(a, b)
        assert same_bits(kept, end)


def test_two_streams_at_once(dev):
    """Calls that overlap in time, each with its own workspace, do not meet."""
    t, d, vocab = torch.bfloat16, 256, 3000
    x, w = randn((600, d), t, dev, 1), randn((vocab, d), t, dev, 2, 0.2)
    at = torch.arange(600, device=dev)
    gate = randn((1, 4000, 64), t, dev, 3)
    dl = torch.ones(600, device=dev)

    def run():
        f = det.det_linear_cross_entropy(x, w, at)
        r = det.det_gated_scan(gate, gate, sigmoid=True)
        return [f.loss, *det.det_linear_cross_entropy_backward(x, w, at, f.lse, dl), r.h, r.state,
                det.det_embedding_backward(x, at, vocab)]

    want = run()
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(run())
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, want):
            assert same_bits(a, b)
