"""det_linear_cross_entropy and its gradients on the GPU against 64-bit statements, at sizes around
the tiles (256 by 256, 64 steps of k), odd widths and offsets, and what holds bit for bit.

Tolerances: a logit is a sum of d products; each addition is off by at most a whole step 2^-23 of the
running sum (matrix instructions), so z is off by ez = (d + 8) 2^-23 sum|x||w| scale; f32 adds 2^-21 of
the same sum (three parts: 2^-24 for each of the products left out, and the six partial sums).  lse is
off by the largest ez, the exponentials (2 (1 + |z - lse|) U each) and sums of up to 16 * 4 + 6 + 2 +
tiles / 64 + 6 terms.  D is off by p times that, by |lse| U, and its rounding; the gradients are sums of
those and of D's products."""
import pytest
import torch

import recurrent_reference as ref
from lm_reference import IDS, TYPES, U32, floor_of, half, randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -23


def inputs(rows, vocab, d, t, dev, seed):
    x = randn((rows, d), t, dev, seed)
    w = randn((vocab, d), t, dev, seed + 1, 2.5 / d ** 0.5)
    at = torch.randint(0, vocab, (rows,), device=dev, generator=torch.Generator(dev).manual_seed(seed))
    if rows > 2:
        at[1], at[rows - 1] = -100, vocab
    return x, w, at


def logit_error(d, t, size):
    return ((d + 8) * STEP + (2.0 ** -21 if t == torch.float32 else 0.0)) * size


SIZES = [(1, 1, 1), (1, 3, 8), (5, 7, 3), (3, 255, 64), (2, 256, 65), (4, 257, 128), (33, 300, 100),
         (64, 513, 72), (65, 700, 40), (130, 1000, 257), (256, 511, 64), (257, 256, 200), (300, 5001, 96),
         (70, 9000, 136), (1, 20000, 512), (17, 4097, 1000)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab,d", SIZES)
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_loss_and_gradients(dev, rows, vocab, d, t, scale):
    x, w, at = inputs(rows, vocab, d, t, dev, rows + d)
    got = det.det_linear_cross_entropy(x, w, at, scale)
    loss, lse, z, size = ref.xent(x, w, at, scale)
    ez = logit_error(d, t, size)
    log = (z - lse[:, None]).abs()
    p = torch.exp(z - lse[:, None])
    terms = 16 * 4 + 16 + vocab / 256 / 64
    rel = (p * (ez + 4 * (1 + log) * U32)).sum(1) + terms * U32
    el = rel * 1.01 + 4 * U32 * (1 + (lse - z.amax(1)).abs()) + 2 * U32 * lse.abs() + U32 * z.amax(1).abs()
    assert ((got.lse.double() - lse).abs() <= el).all()
    on = (at >= 0) & (at < vocab)
    eloss = torch.where(on, el + ez.amax(1) + 2 * U32 * loss.abs(), 0.0)
    assert ((got.loss.double() - loss).abs() <= eloss).all()

    dl = randn((rows,), torch.float32, dev, 4)
    dx, dw = det.det_linear_cross_entropy_backward(x, w, at, got.lse, dl, scale)
    wx, ww, dd, f = ref.xent_backward(x, w, at, got.lse, dl, scale)
    ed = p * (ez + el[:, None] + (2 * lse.abs()[:, None] + 4 * (1 + log)) * U32) * 1.01 + 2 * U32 * (dd.abs() + p)
    # D's storage: its half step; f16 holds D * 2^14
    ed = ed + 1.01 * half(t) * dd.abs() + (2.0 ** -39 if t == torch.float16 else 2.0 ** -126)
    small = f.abs().amax() * 2.0 ** -38 if t == torch.float16 else 0.0      # dweight's D: times dloss / max
    ed = torch.where(on[:, None], ed, 0.0)
    sums = (vocab + 16) * STEP + (2.0 ** -20 if t == torch.float32 else 0.0)
    ex = f.abs() * (ed @ w.double().abs() + sums * (dd.abs() @ w.double().abs()))
    assert ((dx.double() - wx).abs() <= ex * 1.01 + half(t) * (wx.abs() + ex) * 1.01 + floor_of(t)).all()
    sums = (rows + 80) * STEP + (2.0 ** -20 if t == torch.float32 else 0.0)
    xa = x.double().abs()
    ew = (ed * f.abs() * (1 + half(t)) + half(t) * (dd * f).abs() * 1.01 + small).t() @ xa
    ew = ew + sums * ((dd * f).abs().t() @ xa) + 4 * U32 * ww.abs()
    assert ((dw.double() - ww).abs() <= ew * 1.01 + half(t) * (ww.abs() + ew) * 1.01 + floor_of(t)).all()
    off = ~on
    assert (dx[off] == 0).all() and (got.loss[off] == 0).all()


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab,d", [(5, 300, 64), (90, 9001, 72), (300, 4500, 136)])
def test_views_repeats_and_places_keep_their_bits(dev, rows, vocab, d, t):
    x, w, at = inputs(rows, vocab, d, t, dev, 3)
    dl = randn((rows,), torch.float32, dev, 4)

    def both(a, b):
        f = det.det_linear_cross_entropy(a, b, at, 1.25)
        return [*f, *det.det_linear_cross_entropy_backward(a, b, at, f.lse, dl, 1.25)]

    want = both(x, w)
    for a, b in zip(want, both(x, w)):
        assert same_bits(a, b)
    # rows at odd addresses and strides: laid out first, the same sums
    wx = torch.full((rows, d + 9), float("nan"), device=dev).to(t)
    ww = torch.full((vocab, d + 5), float("nan"), device=dev).to(t)
    wx[:, 1:d + 1], ww[:, 3:d + 3] = x, w
    for a, b in ((wx[:, 1:d + 1], w), (x, ww[:, 3:d + 3]), (wx[:, 1:d + 1], ww[:, 3:d + 3])):
        for u, v in zip(want, both(a, b)):
            assert same_bits(u, v)
    # rows with room behind them, on 16 bytes
    wx, ww = torch.full((rows, d + 24), float("nan"), device=dev).to(t), torch.zeros(vocab, d + 40, device=dev).to(t)
    wx[:, :d], ww[:, 8:d + 8] = x, w
    for u, v in zip(want, both(wx[:, :d], ww[:, 8:d + 8])):
        assert same_bits(u, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = both(x, w)
    torch.cuda.current_stream().wait_stream(s)
    for u, v in zip(want, other):
        assert same_bits(u, v)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_rows_that_are_not_scored(dev, t):
    """Whatever they hold, they add nothing; scored rows of infinity and NaN stay alone in dx."""
    x, w, at = inputs(40, 600, 72, t, dev, 9)
    at[5:9] = -1
    clean = det.det_linear_cross_entropy(x, w, at)
    dl = randn((40,), torch.float32, dev, 1)
    want = det.det_linear_cross_entropy_backward(x, w, at, clean.lse, dl)
    junk, jl = x.clone(), dl.clone()
    junk[5], junk[6], junk[7, 3] = float("nan"), float("inf"), float("-inf")
    jl[5:8] = float("nan")
    got = det.det_linear_cross_entropy(junk, w, at)
    keep = torch.arange(40, device=dev) < 5
    assert same_bits(got.loss, clean.loss) and same_bits(got.lse[keep], clean.lse[keep])
    back = det.det_linear_cross_entropy_backward(junk, w, at, got.lse, jl)
    assert same_bits(back[0], want[0]) and same_bits(back[1], want[1])
    junk[20, 1] = float("nan")
    got = det.det_linear_cross_entropy(junk, w, at)
    assert got.loss[20].isnan() and same_bits(got.loss[:20], clean.loss[:20])
    dx = det.det_linear_cross_entropy_backward(junk, w, at, got.lse, jl)[0]
    rows = [i for i in range(40) if i != 20]
    assert same_bits(dx[rows], want[0][rows]) and dx[20].isnan().any()


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_confident_rows_and_far_logits(dev, t):
    """One logit takes all the mass; logits of hundreds."""
    d, vocab = 64, 700
    x, w, at = inputs(9, vocab, d, t, dev, 2)
    x = (40 * w[at.clamp(0, vocab - 1)].float()).to(t)
    got = det.det_linear_cross_entropy(x, w, at)
    loss, lse, z, size = ref.xent(x, w, at, 1.0)
    ez = logit_error(d, t, size).amax(1) + 100 * U32 + 2 * U32 * lse.abs()
    assert ((got.loss.double() - loss).abs() <= 2 * ez).all() and (got.loss >= 0).all()
    dl = torch.ones(9, device=dev)
    dx, dw = det.det_linear_cross_entropy_backward(x, w, at, got.lse, dl)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("small", [2.0 ** -30, 1.0, 3e4])
def test_f16_gradients_of_small_and_large_losses(dev, small):
    """Factors of the loss far from f16's exponents: D is held apart from them."""
    t, rows, vocab, d = torch.float16, 60, 3000, 64
    x, w, at = inputs(rows, vocab, d, t, dev, 2)
    f = det.det_linear_cross_entropy(x, w, at)
    dl = torch.full((rows,), small, device=dev)
    dx, dw = det.det_linear_cross_entropy_backward(x, w, at, f.lse, dl)
    wx, ww, _, _ = ref.xent_backward(x, w, at, f.lse, dl, 1.0)
    for got, want in ((dx, wx), (dw, ww)):
        # values from 65520 on round to infinity
        fits, over = want.abs() < 65520 * (1 - 2e-3), want.abs() > 65520 * (1 + 2e-3)
        assert (got[over].double() == torch.sign(want[over]) * float("inf")).all()
        off = (got.double() - want)[fits]
        assert off.norm() <= 2e-3 * want[fits].norm() + 2.0 ** -25 * want.numel() ** 0.5


def test_no_rows_and_leading_dimensions(dev):
    t = torch.bfloat16
    x, w, at = inputs(12, 90, 32, t, dev, 6)
    none = det.det_linear_cross_entropy(x[:0], w, at[:0])
    assert none.loss.shape == (0,)
    dx, dw = det.det_linear_cross_entropy_backward(x[:0], w, at[:0], none.lse, none.loss)
    assert dx.shape == (0, 32) and dw.shape == w.shape and (dw == 0).all()
    flat = det.det_linear_cross_entropy(x, w, at)
    deep = det.det_linear_cross_entropy(x.view(3, 4, 32), w, at.view(3, 4))
    assert deep.loss.shape == (3, 4) and same_bits(deep.loss.view(-1), flat.loss)
    one = det.det_linear_cross_entropy(x[0], w, at[0])
    assert one.loss.shape == ()
    for bad in (lambda: det.det_linear_cross_entropy(x, w[:0], at),
                lambda: det.det_linear_cross_entropy(x[:, :0], w[:, :0], at)):
        with pytest.raises(det.DetError):
            bad()


def test_gradient_against_differences(dev):
    x, w, at = inputs(9, 300, 24, torch.float32, dev, 7)
    a, b = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    c = randn((9,), torch.float32, dev, 8)
    (det.linear_cross_entropy(a, b, at, 1.5) * c).sum().backward()

    def value(u, v):
        return float((ref.xent(u, v, at, 1.5)[0] * c.double()).sum())

    args = [x.double(), w.double()]
    for n, v in enumerate((a, b)):
        step = randn(v.shape, torch.float32, dev, 30 + n).double()
        lo, hi = list(args), list(args)
        e = 1e-5
        lo[n], hi[n] = args[n] - e * step, args[n] + e * step
        slope = (value(*hi) - value(*lo)) / (2 * e)
        got = float((v.grad.double() * step).sum())
        size = float((v.grad.double() * step).abs().sum())
        assert abs(got - slope) <= 1e-5 * size + 1e-6, (n, got, slope)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab,d", [(3, 70001, 8), (40, 66000, 5), (150, 131100, 12), (1100, 61500, 8)])
def test_vocabularies_of_several_pieces(dev, rows, vocab, d, t):
    test_loss_and_gradients(dev, rows, vocab, d, t, 1.0)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_loss_gradient_that_is_not_finite_shows(dev, t, bad):
    """In its own row of dx, and in all that it adds to."""
    x, w, at = inputs(20, 300, 16, t, dev, 2)
    at[3] = 5
    f = det.det_linear_cross_entropy(x, w, at)
    dl = torch.ones(20, device=dev)
    dl[3] = bad
    dx, dw = det.det_linear_cross_entropy_backward(x, w, at, f.lse, dl)
    assert not torch.isfinite(dx[3]).any() and torch.isfinite(torch.cat([dx[:3], dx[4:]])).all()
    assert not torch.isfinite(dw).any()
