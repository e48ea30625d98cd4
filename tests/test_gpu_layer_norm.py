"""det_layer_norm and its backward pass on the GPU against 64-bit statements, and what holds bit for
bit: repeats, rows alone and among others, views at odd offsets, work in place.

Tolerances: U = 2^-24 is half a step of f32.  A row's sum of d terms is a chain of at most 8 * 4 terms
a lane (8 * d / 8192 past 16384), 6 tree levels and 16 wave sums: `chain`.  The mean is off by em =
(chain + 2) U mean|h|, the distance h - mean by em and its own rounding, the variance's root by half
of (chain + 4) U plus em's share."""
import pytest
import torch

import recurrent_reference as ref
from lm_reference import IDS, TYPES, U32, floor_of, half, randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu
EPS = 1e-5


def chain(d):
    return 8 * max(4, -(-d // 8192)) + 6 + 16


def inputs(rows, d, t, dev, seed, residual=True, bias=True):
    size = torch.exp(0.5 * randn((d,), torch.float32, dev, seed))
    x = ((randn((rows, d), torch.float32, dev, seed + 1) + 0.5) * size).to(t)
    r = (randn((rows, d), torch.float32, dev, seed + 2) * size).to(t) if residual else None
    w = (1 + 0.2 * randn((d,), torch.float32, dev, seed + 3)).to(t)
    return x, r, w, randn((d,), t, dev, seed + 4, 0.1) if bias else None


SIZES = [(1, 1), (3, 2), (3, 7), (5, 64), (2, 511), (4, 512), (3, 513), (2, 1024), (3, 1031), (2, 2048),
         (2, 2049), (3, 4096), (2, 4097), (2, 5001), (2, 6145), (1, 8192), (2, 8193), (2, 16384),
         (2, 16385), (1, 40001)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_layer_norm(dev, rows, d, t, residual):
    x, r, w, b = inputs(rows, d, t, dev, d, residual, bias=d % 3 != 0)
    got = det.det_layer_norm(x, w, b, eps=EPS, residual=r)
    h, mean, rstd, y = ref.layer_norm(x, w, b, EPS, r)
    c = chain(d)
    size = x.double().abs() + (r.double().abs() if residual else 0.0)
    if residual:
        assert same_bits(got.h, (x.float() + r.float()).to(t))
    else:
        assert got.h is x
    em = (c + 3) * U32 * size.mean(1)
    assert ((got.mean.double() - mean).abs() <= em).all()
    dist = (h - mean[:, None]).abs()
    off = em[:, None] + U32 * size + U32 * dist      # of a distance
    # sum of squares: 2 e off + off^2, and its own roundings
    square = (2 * dist * off + off * off).mean(1) * rstd ** 2 + (c + 4) * U32
    er = 0.5 * square * 1.001 + 4 * U32
    assert ((got.rstd.double() - rstd).abs() <= er * rstd).all()
    rw = rstd[:, None] * w.double().abs()
    bound = rw * off + dist * rw * (er[:, None] + 4 * U32) + 2 * U32 * y.abs()
    bound = bound * 1.001 + half(t) * (y.abs() + bound) + floor_of(t)
    assert ((got.y.double() - y).abs() <= bound).all()


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_rows_far_from_zero_keep_their_variance(dev, t):
    """A mean of hundreds of steps of the type and a spread of a few of them."""
    base = {torch.float32: 1000.0, torch.float16: 100.0, torch.bfloat16: 16.0}[t]
    x = (base + randn((5, 700), torch.float32, dev, 3)).to(t)
    w = torch.ones(700, device=dev).to(t)
    got = det.det_layer_norm(x, w, eps=0.0)
    _, mean, rstd, y = ref.layer_norm(x, w, None, 0.0)
    off = (chain(700) + 4) * U32 * base * 1.1
    assert ((got.y.double() - y).abs() <= 2 * off * rstd[:, None] + (half(t) + 64 * U32) * y.abs() + off).all()


def test_constant_rows_and_non_finite_rows(dev):
    x, r, w, b = inputs(6, 700, torch.float32, dev, 5)
    clean = det.det_layer_norm(x, w, b, residual=r)
    x[1, 3], x[4, 699] = float("nan"), float("inf")
    got = det.det_layer_norm(x, w, b, residual=r)
    for i in (0, 2, 3, 5):
        assert same_bits(got.y[i], clean.y[i])
    assert got.y[1].isnan().all() and got.y[4].isnan().all()
    flat = det.det_layer_norm(torch.full((3, 64), 2.0, device=dev), w[:64], b[:64])
    assert same_bits(flat.y, b[:64].expand(3, 64).contiguous()) and (flat.mean == 2).all()
    one = det.det_layer_norm(torch.full((3, 1), 5.0, device=dev), w[:1], b[:1])
    assert (one.y == b[0]).all()


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_rows_of_no_elements_are_refused(dev, t):
    x, w = torch.empty(5, 0, dtype=t, device=dev), torch.empty(0, dtype=t, device=dev)
    s = torch.empty(5, device=dev)
    for call in (lambda: det.det_layer_norm(x, w), lambda: det.layer_norm(x, w),
                 lambda: det.det_layer_norm_backward(x, x, w, s, s)):
        with pytest.raises(det.DetError):
            call()
    none = det.det_layer_norm(torch.empty(0, 0, dtype=t, device=dev), w)
    assert none.y.shape == (0, 0) and none.rstd.shape == (0,)


def test_zero_rows_and_leading_dimensions(dev):
    w = torch.ones(96, device=dev)
    for shape in ((0, 96), (2, 0, 96)):
        got = det.det_layer_norm(torch.empty(shape, device=dev), w, w)
        assert got.y.shape == shape and got.mean.shape == shape[:-1]
        dx, dw, db = det.det_layer_norm_backward(got.y, got.y, w, got.mean, got.rstd)
        assert dx.shape == shape and (dw == 0).all() and (db == 0).all()
    x, r, w, b = inputs(12, 96, torch.bfloat16, dev, 3)
    flat = det.det_layer_norm(x, w, b, residual=r)
    deep = det.det_layer_norm(x.view(3, 4, 96), w, b, residual=r.view(3, 4, 96))
    assert deep.mean.shape == (3, 4) and same_bits(deep.y.view(12, 96), flat.y)
    one = det.det_layer_norm(x[0], w, b, residual=r[0])
    assert one.rstd.shape == () and same_bits(one.y, flat.y[0])


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("d", [96, 1000, 4096, 9000, 17001])
def test_rows_views_and_places_keep_their_bits(dev, d, t):
    x, r, w, b = inputs(37, d, t, dev, d)
    want = det.det_layer_norm(x, w, b, residual=r)
    again = det.det_layer_norm(x, w, b, residual=r)
    alone = det.det_layer_norm(x[11:12], w, b, residual=r[11:12])
    for a, e, c in zip(want, again, alone):
        assert same_bits(a, e) and same_bits(a[11:12], c)
    wide = torch.full((37, d + 9), float("nan"), device=dev).to(t)
    wide[:, 1:d + 1] = x
    shifted = torch.zeros(2, d + 1, device=dev).to(t)
    shifted[0, 1:], shifted[1, 1:] = w, b
    for a, e in zip(want, det.det_layer_norm(wide[:, 1:d + 1], shifted[0, 1:], shifted[1, 1:], residual=r)):
        assert same_bits(a, e)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = det.det_layer_norm(x, w, b, residual=r)
    torch.cuda.current_stream().wait_stream(s)
    assert same_bits(other.y, want.y)
    for replaced in (0, 1):      # h in place of an input
        ins = [x.clone(), r.clone()]
        y, sums = torch.empty_like(x), torch.empty(2, 37, device=dev)
        code = {torch.float32: det.DET_F32, torch.float16: det.DET_F16}.get(t, det.DET_BF16)
        assert det.lib().det_layer_norm(
            ins[0].data_ptr(), d, ins[1].data_ptr(), d, w.data_ptr(), b.data_ptr(), 37, d, code, 1e-5,
            ins[replaced].data_ptr(), y.data_ptr(), sums[0].data_ptr(), sums[1].data_ptr(),
            torch.cuda.current_stream().cuda_stream) == 0
        assert same_bits(ins[replaced], want.h) and same_bits(y, want.y)
        assert same_bits(sums[0], want.mean) and same_bits(sums[1], want.rstd)


BACK = [(1, 1), (3, 7), (9, 64), (2, 512), (7, 513), (5, 2048), (6, 2049), (3, 4096), (5, 5001),
        (2, 8192), (3, 8193), (2, 16384), (9, 16390), (3000, 24), (2100, 520), (1300, 9001)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,d", BACK)
@pytest.mark.parametrize("stream", [False, True])
def test_layer_norm_backward(dev, rows, d, t, stream):
    x, r, w, b = inputs(rows, d, t, dev, d + rows)
    f = det.det_layer_norm(x, w, b, residual=r)
    dy = randn((rows, d), t, dev, 77, 1e-2)
    dh = randn((rows, d), t, dev, 78, 1e-2) if stream else None
    bias = (rows + d) % 2 == 0
    dx, dw, db = det.det_layer_norm_backward(dy, f.h, w, f.mean, f.rstd, dh, bias=bias)
    want, dwant, bwant = ref.layer_norm_backward(dy, f.h, w, f.mean, f.rstd, dh)
    rs = f.rstd.double()[:, None]
    xhat = ((f.h.double() - f.mean.double()[:, None]) * rs).abs()
    g = (dy.double() * w.double()).abs()
    # the row's sums: chains of (chain + 4) roundings of terms of these magnitudes
    terms = rs * (g + g.mean(1, keepdim=True) + xhat * (g * xhat).mean(1, keepdim=True))
    bound = (chain(d) + 14) * U32 * terms + half(t) * want.abs() * 1.001 + floor_of(t)
    if stream:
        bound += 2 * U32 * dh.double().abs()
    assert ((dx.double() - want).abs() <= bound).all()
    # the rows' sums: a strip of at most 8 rows here, the strips of a workgroup and of a lane, the
    # levels above
    depth = 8 + -(-rows // 64) + 6 + 5
    for got, exact, mags in ((dw, dwant, (dy.double().abs() * xhat).sum(0)),
                             (db, bwant, dy.double().abs().sum(0))):
        if got is not None:
            assert ((got.double() - exact).abs() <= depth * U32 * mags
                    + half(t) * exact.abs() * 1.001 + floor_of(t)).all()
    assert (db is not None) == bias
    again = det.det_layer_norm_backward(dy, f.h, w, f.mean, f.rstd, dh, bias=bias)
    assert same_bits(again[0], dx) and same_bits(again[1], dw)
    other = det.det_layer_norm_backward(dy, f.h, w, f.mean, f.rstd, dh, bias=not bias)
    assert same_bits(other[0], dx) and same_bits(other[1], dw)      # with or without the other sum
    i = rows // 2
    alone = det.det_layer_norm_backward(dy[i:i + 1], f.h[i:i + 1], w, f.mean[i:i + 1], f.rstd[i:i + 1],
                                        None if dh is None else dh[i:i + 1])
    assert same_bits(alone[0], dx[i:i + 1])


def test_layer_norm_backward_strided_and_in_place(dev):
    t, rows, d = torch.float16, 11, 777
    x, r, w, b = inputs(rows, d, t, dev, 9)
    f = det.det_layer_norm(x, w, b, residual=r)
    dy, dh = randn((rows, d), t, dev, 1, 1e-2), randn((rows, d), t, dev, 2, 1e-2)
    want = det.det_layer_norm_backward(dy, f.h, w, f.mean, f.rstd, dh)
    wide = torch.zeros(3, rows, d + 5, dtype=t, device=dev)
    for i, v in enumerate((dy, f.h, dh)):
        wide[i, :, 3:3 + d] = v
    got = det.det_layer_norm_backward(wide[0, :, 3:3 + d], wide[1, :, 3:3 + d], w, f.mean, f.rstd,
                                      wide[2, :, 3:3 + d])
    for a, e in zip(got, want):
        assert same_bits(a, e)
    for i in range(3):
        ins = [dy.clone(), f.h.clone(), dh.clone()]
        dw, db = torch.empty_like(w), torch.empty_like(w)
        ws = torch.empty(det.det_layer_norm_backward_workspace_size(rows, d, det.DET_F16),
                         dtype=torch.uint8, device=dev)
        assert det.lib().det_layer_norm_backward(
            ins[0].data_ptr(), d, ins[1].data_ptr(), d, w.data_ptr(), f.mean.data_ptr(),
            f.rstd.data_ptr(), ins[2].data_ptr(), d, rows, d, det.DET_F16, ins[i].data_ptr(),
            dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream) == 0
        assert same_bits(ins[i], want[0]) and same_bits(dw, want[1]) and same_bits(db, want[2])


@pytest.mark.parametrize("d", [5, 300, 2100])
def test_gradient_against_differences(dev, d):
    x, r, w, b = inputs(4, d, torch.float32, dev, 21)
    for v in (x, r, w, b):
        v.requires_grad_(True)
    y, h = det.layer_norm(x, w, b, r)
    cy, ch = randn((4, d), torch.float32, dev, 22), randn((4, d), torch.float32, dev, 23)
    ((y * cy).sum() + (h * ch).sum()).backward()

    def value(a, b, c, e):
        hh, _, _, yy = ref.layer_norm(a, c, e, EPS, b)
        return float((yy * cy.double()).sum() + (hh * ch.double()).sum())

    args = [v.detach().double() for v in (x, r, w, b)]
    for n, v in enumerate((x, r, w, b)):
        step = randn(v.shape, torch.float32, dev, 30 + n).double()
        lo, hi = list(args), list(args)
        e = 1e-5
        lo[n], hi[n] = args[n] - e * step, args[n] + e * step
        slope = (value(*hi) - value(*lo)) / (2 * e)
        got = float((v.grad.double() * step).sum())
        # differences: third derivatives times e^2 and the values' rounding over e, 64 bits
        size = float((v.grad.double() * step).abs().sum())
        assert abs(got - slope) <= 1e-5 * size + 1e-6, (n, got, slope)


def test_autograd_paths(dev):
    x, r, w, b = inputs(6, 130, torch.bfloat16, dev, 50)
    f = det.det_layer_norm(x, w, b)
    dy = randn((6, 130), torch.bfloat16, dev, 51)
    want = det.det_layer_norm_backward(dy, x, w, f.mean, f.rstd)
    leaves = [v.clone().requires_grad_(True) for v in (x, w, b)]
    det.layer_norm(*leaves).backward(dy)
    for v, g in zip(leaves, want):
        assert same_bits(v.grad, g)
    a, c = x.clone().requires_grad_(True), r.clone().requires_grad_(True)
    _, h = det.layer_norm(a, w, None, c)
    h.backward(dy)      # only h is used further: the norm's own part is zero
    assert torch.equal(a.grad, dy) and torch.equal(c.grad, dy)
    a = x.clone().requires_grad_(True)
    det.layer_norm(a, w, b).sum().backward()      # a broadcast gradient
    assert same_bits(a.grad, det.det_layer_norm_backward(torch.ones_like(x), x, w, f.mean, f.rstd)[0])
