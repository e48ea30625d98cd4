"""Edges of the language-model operators on the GPU: rows of no elements, values at the ends of
their types, sizes at the ends of a launch."""
import math

import pytest
import torch

import lm_reference as ref
from lm_reference import IDS, TYPES, U32, floor_of, half, randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_rows_of_no_elements_are_refused(dev, t):
    # rstd and scales would have five values that nothing gives
    x, w = torch.empty(5, 0, dtype=t, device=dev), torch.empty(0, dtype=t, device=dev)
    rstd = torch.empty(5, device=dev)
    for call in (lambda: det.det_rms_norm(x, w), lambda: det.det_rms_norm(x, w, quant=E4M3),
                 lambda: det.det_rms_norm(x, w, residual=x), lambda: det.rms_norm(x, w),
                 lambda: det.det_rms_norm_backward(x, x, w, rstd)):
        with pytest.raises(det.DetError):
            call()
    # no rows at all are no error
    none = det.det_rms_norm(torch.empty(0, 0, dtype=t, device=dev), w, quant=E4M3)
    assert none.y.shape == (0, 0) and none.rstd.shape == (0,) and none.scales.shape == (0, 1)


# ------------------------------------------------------------------ rows far from zero

def gradient_bound(x, at, scale, dlogp, dentropy, want, t):
    """Against the gradient of the logits alone (no lse handed in): log p is off by its own
    roundings and by the sum's relative error `rel` (chains of vocab / 256 terms and more, each
    term off by 2 U (1 + |z - max|)), or by the rounding of an lse of at most 256."""
    _, entropy, lse, log = ref.logprobs(x, at, scale)
    p, size = log.exp(), torch.where(log > -math.inf, log.abs(), 0.0)
    far = (p * size).sum(-1, keepdim=True) + 8
    rel = U32 * (40 + x.shape[-1] / 256 + 4 * far + lse.abs().clamp_max(256.0)[:, None])
    d, e = dlogp.double().abs()[:, None], dentropy.double().abs()[:, None]
    hit = torch.zeros_like(p).scatter_(1, at.clamp_min(0)[:, None], 1.0)
    parts = d * (hit + p) + e * p * (size + entropy[:, None])
    bound = ((8 + 4 * size) * U32 + rel) * parts + e * p * rel * (2 + far)
    bound += 2.0 ** -126 * (d + e + 1) * (1 + size.clamp_max(200.0))
    return bound * scale + half(t) * want.abs() * 1.001 + floor_of(t)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("vocab", [5, 1000, 9001, 20003])
@pytest.mark.parametrize("scale", [1.0, 0.5])
def test_gradient_of_rows_far_from_zero(dev, vocab, t, scale):
    """lse is a float, and log(sum) is lost in it where the logits are large: in a row of the type's
    lowest values (a mask that leaves nothing) altogether."""
    low = torch.finfo(t).min
    x = randn((9, vocab), torch.float32, dev, 31, 2.0)
    for i, off in enumerate((0.0, 200.0, -300.0, 700.0, -6000.0, 50000.0)):
        x[i] += off
    x = x.to(t)
    x[6] = low
    x[7, vocab // 2:] = low
    x[8] = low
    x[8, 1] = -math.inf
    x[3, ::2] = -math.inf
    at = torch.arange(9, device=dev) % vocab
    at[5] = -100
    dlogp, dent = randn((9,), torch.float32, dev, 32), randn((9,), torch.float32, dev, 33)
    dlogp_in = torch.where(at >= 0, dlogp, 0.0)
    f = det.det_token_logprobs(x, at, scale)
    got = det.det_token_logprobs_backward(x, at, f.lse, dlogp, f.entropy, dent, scale)
    _, entropy, _, log = ref.logprobs(x, at, scale)
    want = ref.logprobs_backward(log, at, entropy, dlogp, dent, scale)
    assert ((got.double() - want).abs()
            <= gradient_bound(x, at, scale, dlogp_in, dent, want, t)).all()
    # each row alone, in place, and among padded columns: the same bits
    for i in range(9):
        one = det.det_token_logprobs_backward(x[i:i + 1], at[i:i + 1], f.lse[i:i + 1],
                                              dlogp[i:i + 1], f.entropy[i:i + 1], dent[i:i + 1], scale)
        assert same_bits(one, got[i:i + 1])
    again = x.clone()
    det.det_token_logprobs_backward(again, at, f.lse, dlogp, f.entropy, dent, scale, out=again)
    assert same_bits(again, got)
    wide = torch.zeros(9, vocab + 5, dtype=t, device=dev)
    wide[:, 2:vocab + 2] = x
    assert same_bits(det.det_token_logprobs_backward(wide[:, 2:vocab + 2], at, f.lse, dlogp,
                                                     f.entropy, dent, scale), got)
    v = x.clone().requires_grad_(True)
    logp, ent = det.token_logprobs(v, at, scale)
    ((logp * dlogp).sum() + (ent * dent).sum()).backward()
    assert same_bits(v.grad, got)


# ------------------------------------------------------------------ not a number

NANS = {torch.float32: (torch.int32, (0x7F800001, 0x7FA00000, 0x7FC00000, -0x7FFFFF, -1)),
        torch.float16: (torch.int16, (0x7C01, 0x7D00, 0x7E00, -0x3FF, -1)),
        torch.bfloat16: (torch.int16, (0x7F81, 0x7FA0, 0x7FC0, -0x7F, -1))}


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab", [(3, 70), (8, 9001), (300, 9001), (600, 9001), (4, 40000)])
def test_alternatives_beside_a_signalling_nan(dev, rows, vocab, t):
    """Every kind of NaN counts as -inf among the alternatives, wherever it stands beside the best."""
    kind, bits = NANS[t]
    x = randn((rows, vocab), torch.float32, dev, 41).to(t)
    best = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(1))
    for i in range(rows):
        x[i, best[i]] = 40.0
    raw = x.view(kind)
    for i in range(rows):
        for j, step in enumerate((-31, -9, -4, -1, 1, 2, 3, 7, 16)[:5 + i % 5]):
            p = int(best[i]) + step
            if 0 <= p < vocab:
                raw[i, p] = bits[(i + j) % len(bits)]
    raw[0] = bits[0]                                  # nothing else at all
    raw[1, ::2] = bits[1]
    nan = x.isnan()
    assert nan[0].all() and nan.any(1).all()
    at = torch.zeros(rows, dtype=torch.int64, device=dev)
    got = det.det_token_logprobs(x, at, top=20)
    want = ref.top_ids(torch.where(nan, -math.inf, x.double()), 20)
    assert torch.equal(got.top_ids, want)
    assert got.lse.isnan().all() and got.logp.isnan().all() and got.entropy.isnan().all()


# ------------------------------------------------------------------ rows of one likely token

@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("first,second", [(0, 40960), (40960, 0), (3, 9), (17, 700), (4999, 33)])
@pytest.mark.parametrize("top", [0, 2])
def test_likely_tokens_keep_their_digits(dev, first, second, top, t):
    """Two tokens, `gap` apart: s = 1 + r with r = exp(-gap).  r is off by (2 gap + 4) U (product
    with log2 e and its constant, the hardware's unit, one rescaling), the sum by U, the logarithm
    by two half-steps; the entropy's second term gap r / s by the same and three more roundings."""
    gap = torch.arange(1, 129, device=dev) / 8
    x = torch.full((128, 50000), -math.inf, device=dev)
    x[:, first] = -3.0
    x[:, second] = gap - 3.0
    x = x.to(t)
    gap = x[:, second].double() - x[:, first].double()
    at = torch.full((128,), second, device=dev)
    got = det.det_token_logprobs(x, at, top=top)
    r = (-gap).exp()
    logp, part = -torch.log1p(r), gap * r / (1 + r)
    off = (1 + r * (2 * gap + 4)) / (1 + r) + 2 * logp.abs()
    assert ((got.logp.double() - logp).abs() <= off * U32).all()
    off = off + part * (2 * gap + 8) + 2 * (part - logp)
    assert ((got.entropy.double() - (part - logp)).abs() <= off * U32).all()
    if top:
        assert torch.equal(got.top_ids, torch.tensor([[second, first]], device=dev).expand(128, 2))
        assert same_bits(got.top_logp[:, 0].contiguous(), got.logp)


# ------------------------------------------------------------------ long rows

@pytest.mark.parametrize("rows,d", [(1, (1 << 26) + 17), (2, (1 << 25) + 1)])
def test_norm_backward_of_the_longest_rows(dev, rows, d):
    """Columns past what one launch of the column sums covers (2^21 workgroups of 16)."""
    h, dy = randn((rows, d), torch.float32, dev, 51), randn((rows, d), torch.float32, dev, 52)
    w = randn((d,), torch.float32, dev, 53)
    rstd = h.double().square().mean(1).rsqrt().float()
    dx, dw = det.det_rms_norm_backward(dy, h, w, rstd)
    # at most two strips of one row each and the tree's zeros: one addition
    terms = dy * (h * rstd[:, None])
    assert torch.equal(dw, terms[0] if rows == 1 else terms[0] + terms[1])
    want, _ = ref.norm_backward(dy, h, w, rstd)
    # a lane's chain of d / 1024 terms, the tree's 10 levels; xhat's mean is small beside dy w
    g, xhat = (dy.double() * w.double()).abs(), (h.double() * rstd.double()[:, None]).abs()
    chain = d / 1024 + 26
    mean = (g * xhat).mean(1, keepdim=True)
    bound = U32 * rstd.double()[:, None] * (8 * (g + xhat * mean) + chain * xhat * mean)
    assert ((dx.double() - want).abs() <= bound).all()


# ------------------------------------------------------------------ the table's gradient in f32

@pytest.mark.parametrize("shape", [(2, 3, 9, 20), (1, 4, 100, 1000), (3, 5, 777, 1003), (2, 8, 1500, 2100)])
@pytest.mark.parametrize("causal", [False, True])
def test_table_gradient_of_f32_is_rounded_once(dev, shape, causal):
    """Sums in double throughout: chains of less than 2^14 terms of 2^-53 each stay below 2^-38 of
    the summed magnitudes, and the result is rounded to float."""
    b, h, q, k = shape
    lens = torch.tensor([k - 3 * i for i in range(b)], dtype=torch.int32, device=dev)
    dout = randn(shape, torch.float32, dev, 61)
    maps = ref.bias_maps(b, q, k, 32, 128, True, causal, k - q, lens.tolist(), dev)
    got = det.det_relative_bias_backward(dout, 32, causal=causal, q_offset=k - q, lengths=lens)
    want, sizes, _ = ref.bias_backward(dout, maps, 32)
    assert ((got.double() - want).abs() <= U32 * want.abs() * 1.001 + 2.0 ** -38 * sizes).all()


# ------------------------------------------------------------------ masks that are numbers

@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab", [(12, 5), (12, 258), (12, 9001), (12, 40000), (300, 9001),
                                        (600, 9001)])
@pytest.mark.parametrize("scale", [1.0, 0.7, 1.25, 3.0, 0.0078125])
def test_masks_of_large_numbers(dev, rows, vocab, t, scale):
    """Logits masked by large negative numbers instead of -inf, under a scale: rows keep their
    values, and rows of nothing else are even."""
    low = torch.finfo(t).min
    masks = [low, low / 1.5, -6e4, -3e4] + ([-1e30, -1e9] if t != torch.float16 else [-5e4, -1e4])
    scale = float(torch.tensor(scale, dtype=torch.float32))
    x = randn((rows, vocab), torch.float32, dev, 71, 2.0).to(t)
    column = torch.arange(vocab, device=dev)
    for i, m in enumerate(masks):
        x[2 * i] = m                                          # nothing is left
        x[2 * i + 1] = torch.where(column % 5 == i % 5, x[2 * i + 1], m)
    at = (column[:1] + torch.arange(rows, device=dev)) % vocab
    top = min(vocab, 7)
    got = det.det_token_logprobs(x, at, scale, top)
    logp, entropy, lse, log = ref.logprobs(x, at, scale)
    p, size = log.exp(), torch.where(log > -math.inf, log.abs(), 0.0)
    far = (p * torch.where(p > 0, size, 0.0)).sum(-1) + 8
    rel = U32 * (40 + vocab / 1024 + 4 * far)
    fits = lse.abs() <= torch.finfo(torch.float32).max
    assert ((got.lse.double() - lse).abs() <= rel + 2 * U32 * lse.abs())[fits].all()
    assert (got.lse[~fits] == -math.inf).all()
    # a masked target's log probability may lie past the floats
    lost = logp < -1e38
    assert (got.logp[lost] < -9e37).all()
    assert ((got.logp.double() - logp).abs() <= rel + 4 * U32 * (logp.abs() + 8))[~lost].all()
    assert ((got.entropy.double() - entropy).abs() <= rel * (2 + far)).all()
    assert torch.equal(got.top_ids, ref.top_ids(x, top))

    dlogp, dent = randn((rows,), torch.float32, dev, 72), randn((rows,), torch.float32, dev, 73)
    grad = det.det_token_logprobs_backward(x, at, got.lse, dlogp, got.entropy, dent, scale)
    want = ref.logprobs_backward(log, at, entropy, dlogp, dent, scale)
    assert ((grad.double() - want).abs()
            <= gradient_bound(x, at, scale, dlogp, dent, want, t)).all()
