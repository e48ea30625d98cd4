"""The language-model operators captured into one graph and replayed on changed inputs, with eager
work between the replays: every replay has the bits of direct calls."""
import pytest
import torch

from lm_reference import randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu


def test_replays_match_direct_calls(dev):
    t, rows, d, vocab, heads, q = torch.bfloat16, 48, 640, 9001, 4, 48
    x, w = randn((rows, d), t, dev, 1), randn((d,), t, dev, 2)
    r, dy = randn((rows, d), t, dev, 3), randn((rows, d), t, dev, 4)
    logits = randn((rows, vocab), t, dev, 5, 2.0)
    at = torch.arange(rows, device=dev) * 100
    dlp = randn((rows,), torch.float32, dev, 6)
    table, scores = randn((32, heads), t, dev, 7), randn((2, heads, q, 333), t, dev, 8)
    lens = torch.tensor([333, 41], dtype=torch.int32, device=dev)

    def run():
        n = det.det_rms_norm(x, w, residual=r)
        c = det.det_rms_norm(x, w, quant=torch.float8_e4m3fn, group=64)
        back = det.det_rms_norm_backward(dy, n.h, w, n.rstd)
        bias = det.det_relative_bias(table, q, 333, scores=scores, causal=True, q_offset=285,
                                     lengths=lens)
        dt = det.det_relative_bias_backward(scores, 32, causal=True, q_offset=285, lengths=lens)
        lp = det.det_token_logprobs(logits, at, top=6)
        dl = det.det_token_logprobs_backward(logits, at, lp.lse, dlp, lp.entropy, dlp)
        return [n.y, n.h, n.rstd, c.y, c.scales, *back, bias, dt, *lp, dl]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for i in range(4):
        for n, v in enumerate((x, r, dy, logits, scores)):
            v.copy_(randn(v.shape, t, dev, 100 * i + n))
        lens.copy_(torch.tensor([333 - i, 50 + i], dtype=torch.int32))
        for o in outs:
            o.view(torch.uint8).fill_(0xA5)
        want = run()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert same_bits(a, b)
