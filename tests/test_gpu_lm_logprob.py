"""det_token_logprobs and its gradient on the GPU against 64-bit statements; the alternatives' ids
have to be equal.

Tolerances: U = 2^-24.  A term exp(z - ref) is off by 2 U (1 + |z - ref|) and the hardware's unit;
terms count by their weight, so with weights p the sums s and w / s are off by U (40 + vocab /
1024 + 4 sum p |z - ref|) relative to s, and by as much times sum p |z - ref| more for w / s.
z - ref and the last additions are rounded once each relative to their sizes."""
import math

import pytest
import torch

import lm_reference as ref
from lm_reference import IDS, TYPES, U32, floor_of, half, randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu


def inputs(rows, vocab, t, dev, seed, spread=2.5):
    x = randn((rows, vocab), torch.float32, dev, seed, spread)
    g = torch.Generator(device=dev)
    g.manual_seed(seed + 1)
    at = torch.randint(0, vocab, (rows,), generator=g, device=dev)
    x[torch.arange(rows, device=dev), at] += 8.0
    at[::5] = -100
    return x.to(t), at


def check(x, at, scale, got, top):
    logp, entropy, lse, log = ref.logprobs(x, at, scale)
    z = torch.where(log > -math.inf, log + lse[..., None], 0.0)
    p = log.exp()
    far = torch.where(p > 0, p * (lse[..., None] - z).abs(), 0.0).sum(-1) + 8
    rel = U32 * (40 + x.shape[-1] / 1024 + 4 * far)
    assert ((got.lse.double() - lse).abs() <= rel + 2 * U32 * lse.abs()).all()
    ok = (at >= 0) & (at < x.shape[-1])
    assert (got.logp[~ok] == 0).all()
    tol = rel + 4 * U32 * (logp.abs() + 8)
    inf = logp == -math.inf
    assert ((got.logp.double() - logp).abs()[~inf] <= tol[~inf]).all()
    assert (got.logp[inf] == -math.inf).all()
    assert ((got.entropy.double() - entropy).abs() <= rel * (2 + far)).all()
    if top:
        ids = ref.top_ids(x, top)
        assert torch.equal(got.top_ids, ids)
        want = log.gather(-1, ids)
        fin = want > -math.inf
        err = (got.top_logp.double() - want).abs()
        assert (err <= rel[..., None] + 4 * U32 * (want.abs() + 8))[fin].all()
        assert (got.top_logp[~fin] == -math.inf).all()
    else:
        assert got.top_ids is None and got.top_logp is None


SIZES = [(1, 1), (3, 2), (2, 31), (5, 33), (4, 1000), (3, 2047), (2, 8191), (3, 8192), (2, 8193),
         (2, 32768), (2, 40000), (300, 9001), (2, 131072), (1, 262144)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("top,scale", [(0, 1.0), (1, 0.8), (5, 1.0), (20, 1.25), (64, 1.0)])
def test_logprobs(dev, rows, vocab, t, top, scale):
    x, at = inputs(rows, vocab, t, dev, vocab + rows)
    top = min(top, vocab)
    check(x, at, scale, det.det_token_logprobs(x, at, scale, top), top)


def test_largest_vocabulary_with_alternatives(dev):
    x, at = inputs(2, 1 << 20, torch.bfloat16, dev, 3)
    check(x, at, 1.0, det.det_token_logprobs(x, at, 1.0, 64), 64)


def test_vocabulary_past_the_alternatives_limit(dev):
    x, at = inputs(1, (1 << 21) + 3, torch.float16, dev, 4)
    check(x, at, 1.0, det.det_token_logprobs(x, at), 0)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows", [3, 400])
@pytest.mark.parametrize("vocab", [200, 20011])
def test_ties_order_and_masks(dev, rows, vocab, t):
    """Equal logits, ascending and descending rows, both zeros, -inf and lowest values."""
    x, at = inputs(rows, vocab, t, dev, 5)
    x[0] = 1.0                                                # all equal
    x[1] = (torch.arange(vocab, device=dev) / 64).to(t)       # ascending, with ties in 16 bits
    x[2] = torch.where(torch.arange(vocab, device=dev) % 2 == 0, -0.0, 0.0).to(t)
    if rows > 3:
        x[3] = (-torch.arange(vocab, device=dev) / 64).to(t)
        x[4] = randn((vocab,), torch.float32, dev, 6).round().to(t)     # many ties
        x[5, 10:] = -math.inf                                 # fewer finite logits than places
        x[6, :vocab - 7] = -math.inf
        x[7, :vocab - 3] = torch.finfo(t).min
        x[8, ::3] = -math.inf
        x[9] = torch.finfo(t).min
        x[10, 0] = torch.finfo(t).max / 2                     # takes all the mass
        x[11] = -math.inf
        x[11, 77] = -3.0
        at[5:12] = 8
        at[11] = 77
    for scale in (1.0, 0.5):
        check(x, at, scale, det.det_token_logprobs(x, at, scale, 20), 20)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows", [4, 300])
def test_rows_without_mass_and_not_a_number(dev, rows, t):
    x, at = inputs(rows, 9000, t, dev, 7)
    clean = det.det_token_logprobs(x, at, top=4)
    x[0] = -math.inf
    x[2, 5000] = math.nan
    at[0], at[2] = 3, 4
    got = det.det_token_logprobs(x, at, top=4)
    assert got.lse[0] == -math.inf and got.entropy[0] == 0 and got.logp[0] == -math.inf
    assert got.top_ids[0].tolist() == [0, 1, 2, 3] and (got.top_logp[0] == -math.inf).all()
    assert got.lse[2].isnan() and got.logp[2].isnan() and got.entropy[2].isnan()
    assert ((got.top_ids[2] >= 0) & (got.top_ids[2] < 9000)).all()
    for i in (1, 3):
        assert all(same_bits(a[i], b[i]) for a, b in zip(got, clean))
    g = det.det_token_logprobs_backward(x, at, got.lse, torch.ones(rows, device=dev), got.entropy,
                                        torch.ones(rows, device=dev))
    assert (g[0] == 0).all() and g[2].isnan().all() and not g[1].isnan().any()


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_targets_outside_are_not_scored(dev, t):
    x, at = inputs(6, 500, t, dev, 8)
    at[:] = torch.tensor([-1, 500, 1 << 40, -(1 << 40), 0, 499], device=dev)
    got = det.det_token_logprobs(x, at)
    check(x, at, 1.0, got, 0)
    assert (got.logp[:4] == 0).all() and (got.logp[4:] < 0).all()
    ones = torch.ones(6, device=dev)
    g = det.det_token_logprobs_backward(x, at, got.lse, ones)
    assert (g[:4] == 0).all() and (g[4:] != 0).any()


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("vocab", [100, 9001, 70000])
def test_rows_views_and_launches_keep_their_bits(dev, vocab, t):
    # few rows and many rows take different workgroups, and the same order
    x, at = inputs(300, vocab, t, dev, 9)
    want = det.det_token_logprobs(x, at, 1.25, 7)
    for r in ((17, 18), (100, 130)):
        part = det.det_token_logprobs(x[r[0]:r[1]], at[r[0]:r[1]], 1.25, 7)
        assert all(same_bits(a, b[r[0]:r[1]].contiguous()) for a, b in zip(part, want))
    wide = torch.full((300, vocab + 13), 50.0, device=dev).to(t)
    wide[:, 3:vocab + 3] = x
    padded = det.det_token_logprobs(wide[:, 3:vocab + 3], at, 1.25, 7)
    deep = det.det_token_logprobs(x.view(3, 100, vocab), at.view(3, 100), 1.25, 7)
    assert deep.top_ids.shape == (3, 100, 7)
    for a, b, c in zip(want, padded, deep):
        assert same_bits(a, b) and same_bits(a, c.view(a.shape))
    plain = det.det_token_logprobs(x, at, 1.25)
    assert same_bits(plain.lse, want.lse) and same_bits(plain.entropy, want.entropy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = det.det_token_logprobs(x, at, 1.25, 7)
    torch.cuda.current_stream().wait_stream(s)
    assert all(same_bits(a, b) for a, b in zip(want, other))


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("vocab", [9001, 40000])
def test_workgroups_of_every_size_keep_the_bits(dev, vocab, t):
    x, at = inputs(600, vocab, t, dev, 20)
    want = det.det_token_logprobs(x, at, 0.8, 20)
    check(x, at, 0.8, want, 20)
    for a, b in ((0, 100), (40, 420), (599, 600)):
        part = det.det_token_logprobs(x[a:b], at[a:b], 0.8, 20)
        assert all(same_bits(p, w[a:b].contiguous()) for p, w in zip(part, want))


def test_rows_past_32_bit_offsets(dev):
    vocab, far = 5000, (1 << 32) + 24
    buf = torch.empty(far + vocab, dtype=torch.bfloat16, device=dev)
    x, at = inputs(2, vocab, torch.bfloat16, dev, 11)
    rows = buf.as_strided((2, vocab), (far, 1))
    rows.copy_(x)
    want, got = det.det_token_logprobs(x, at, top=3), det.det_token_logprobs(rows, at, top=3)
    assert all(same_bits(a, b) for a, b in zip(want, got))
    d = torch.ones(2, device=dev)
    g = det.det_token_logprobs_backward(x, at, want.lse, d)
    assert det.det_token_logprobs_backward(rows, at, want.lse, d, out=rows) is rows
    assert torch.equal(rows, g)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 7), (4, 1000), (2, 8193), (300, 2049), (2, 50021)])
@pytest.mark.parametrize("scale", [1.0, 0.8])
@pytest.mark.parametrize("dent", [False, True])
def test_backward(dev, rows, vocab, t, scale, dent):
    x, at = inputs(rows, vocab, t, dev, vocab)
    x[0, vocab // 3:vocab // 2] = -math.inf
    f = det.det_token_logprobs(x, at, scale)
    dlogp = randn((rows,), torch.float32, dev, 12)
    dentropy = randn((rows,), torch.float32, dev, 13) if dent else None
    got = det.det_token_logprobs_backward(x, at, f.lse, dlogp, f.entropy, dentropy, scale)
    # the formula for the lse and entropy that were handed in
    log = x.double() * scale - f.lse.double()[:, None]
    want = ref.logprobs_backward(log, at, f.entropy.double(), dlogp, dentropy, scale)
    p, size = log.exp(), torch.where(log > -math.inf, log.abs(), 0.0)
    d = dlogp.double().abs()[:, None]
    hit = torch.zeros_like(p).scatter_(1, at.clamp_min(0)[:, None], 1.0)
    parts = d * (hit + p)
    if dent:
        parts = parts + dentropy.double().abs()[:, None] * p * (size + f.entropy.double()[:, None])
    bound = (8 + 4 * size) * U32 * parts * scale + half(t) * want.abs() * 1.001 + floor_of(t)
    # terms below 2^-126 are dropped
    bound += 2.0 ** -126 * (d * scale + 1) * (1 + size.clamp_max(200.0))
    assert ((got.double() - want).abs() <= bound).all()
    assert (got[log == -math.inf] == 0).all()
    again = x.clone()
    assert det.det_token_logprobs_backward(again, at, f.lse, dlogp, f.entropy, dentropy, scale,
                                           out=again) is again
    assert same_bits(again, got)
    wide = torch.zeros(rows, vocab + 5, dtype=t, device=dev)
    wide[:, 2:vocab + 2] = x
    v = wide[:, 2:vocab + 2]
    assert same_bits(det.det_token_logprobs_backward(v, at, f.lse, dlogp, f.entropy, dentropy,
                                                     scale), got)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("vocab", [1000, 1003, 9001])
def test_gradient_of_many_rows_keeps_its_bits(dev, vocab, t):
    # enough rows for many waves on each unit, and rows that end inside a wave and a vector
    rows = 1500
    x, at = inputs(rows, vocab, t, dev, 18)
    f = det.det_token_logprobs(x, at)
    d = randn((rows,), torch.float32, dev, 19)
    want = ref.logprobs_backward(x.double() - f.lse.double()[:, None], at, f.entropy.double(), d,
                                 None, 1.0)
    p = (x.double() - f.lse.double()[:, None]).exp()
    hit = torch.zeros_like(p).scatter_(1, at.clamp_min(0)[:, None], 1.0)
    size = (x.double() - f.lse.double()[:, None]).abs()
    got = det.det_token_logprobs_backward(x, at, f.lse, d)
    bound = (8 + 4 * size) * U32 * d.double().abs()[:, None] * (hit + p)
    bound += half(t) * want.abs() * 1.001 + floor_of(t)
    bound += 2.0 ** -126 * (d.double().abs()[:, None] + 1) * (1 + size.clamp_max(200.0))
    assert ((got.double() - want).abs() <= bound).all()
    for _ in range(5):
        assert same_bits(det.det_token_logprobs_backward(x, at, f.lse, d), got)
    for r in range(0, rows, 100):
        part = det.det_token_logprobs_backward(x[r:r + 100], at[r:r + 100], f.lse[r:r + 100],
                                               d[r:r + 100])
        assert same_bits(part, got[r:r + 100].contiguous())


def test_empty(dev):
    x, at = torch.empty(0, 50, device=dev), torch.empty(0, dtype=torch.int64, device=dev)
    got = det.det_token_logprobs(x, at, top=3)
    assert got.logp.shape == (0,) and got.top_ids.shape == (0, 3)
    assert det.det_token_logprobs_backward(x, at, got.lse, got.lse).shape == (0, 50)


@pytest.mark.parametrize("scale", [1.0, 1.25])
def test_gradient_against_differences(dev, scale):
    rows, vocab = 5, 37
    x, at = inputs(rows, vocab, torch.float32, dev, 14, 1.0)
    x.requires_grad_(True)
    a, b = randn((rows,), torch.float32, dev, 15), randn((rows,), torch.float32, dev, 16)
    logp, entropy = det.token_logprobs(x, at, scale)
    ((logp * a).sum() + (entropy * b).sum()).backward()

    def value(v):
        lp, en, _, _ = ref.logprobs(v, at, scale)
        return float((lp * a.double()).sum() + (en * b.double()).sum())

    base = x.detach().double()
    step = randn(x.shape, torch.float32, dev, 17).double()
    e = 1e-5
    slope = (value(base + e * step) - value(base - e * step)) / (2 * e)
    got = float((x.grad.double() * step).sum())
    assert abs(got - slope) <= 1e-5 * float((x.grad.double() * step).abs().sum()) + 1e-6


def test_autograd_parts(dev):
    x, at = inputs(7, 300, torch.bfloat16, dev, 18)
    f = det.det_token_logprobs(x, at)
    d = randn((7,), torch.float32, dev, 19)
    zero = torch.zeros(7, device=dev)
    for n, want in ((0, det.det_token_logprobs_backward(x, at, f.lse, d)),
                    (1, det.det_token_logprobs_backward(x, at, f.lse, zero, f.entropy, d))):
        v = x.clone().requires_grad_(True)
        det.token_logprobs(v, at)[n].backward(d)
        assert torch.equal(v.grad, want)
