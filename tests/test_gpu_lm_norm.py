"""det_rms_norm and its backward pass on the GPU against 64-bit statements, and what holds bit for
bit: repeats, rows alone and among others, views at odd offsets, work in place.

Tolerances: U = 2^-24 is half a step of f32.  A row's sum of squares of d terms is a chain of at
most 8 * 3 terms a lane (8 * d / 8192 past 16384), 6 tree levels and 16 wave sums, and rstd halves
a relative error; with the root, the division, two products and the residual's addition y is off
by at most (CHAIN + 8) U relative to |h| rstd |w|, and the type's half step."""
import pytest
import torch

import lm_reference as ref
from lm_reference import IDS, TYPES, U32, floor_of, half, randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu
EPS = 1e-6
E4M3 = torch.float8_e4m3fn


def chain(d):
    return 8 * max(4, -(-d // 8192)) + 6 + 16


def inputs(rows, d, t, dev, seed, residual=True):
    size = torch.exp(0.5 * randn((d,), torch.float32, dev, seed))
    x = (randn((rows, d), torch.float32, dev, seed + 1) * size).to(t)
    r = (randn((rows, d), torch.float32, dev, seed + 2) * size).to(t) if residual else None
    return x, r, (1 + 0.2 * randn((d,), torch.float32, dev, seed + 3)).to(t)


SIZES = [(1, 1), (3, 7), (5, 64), (2, 511), (4, 512), (3, 513), (2, 1024), (3, 1031), (2, 2048),
         (2, 2049), (3, 4096), (2, 4097), (2, 5001), (2, 6145), (1, 8192), (2, 8193), (2, 16384),
         (2, 16385), (1, 40001)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(dev, rows, d, t, residual):
    x, r, w = inputs(rows, d, t, dev, d, residual)
    got = det.det_rms_norm(x, w, eps=EPS, residual=r)
    h, rstd, y = ref.norm(x, w, EPS, r)
    c = (chain(d) + 8) * U32
    if residual:
        exact = (x.float() + r.float()).to(t)
        assert same_bits(got.h, exact)
        size = (x.double().abs() + r.double().abs()) * U32 * rstd[:, None] * w.double().abs()
    else:
        assert got.h is x
        size = 0.0
    assert ((got.rstd.double() - rstd).abs() <= c * rstd).all()
    bound = y.abs() * (half(t) + c) * 1.001 + size + floor_of(t)
    assert ((got.y.double() - y).abs() <= bound).all()
    assert got.scales is None


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 31), (3, 129), (5, 512), (2, 1000), (2, 2048),
                                    (3, 5001), (2, 8192), (1, 16384), (2, 16500)])
def test_norm_8bit(dev, rows, d, t, group):
    x, r, w = inputs(rows, d, t, dev, d + group)
    got = det.det_rms_norm(x, w, eps=EPS, residual=r, quant=E4M3, group=group)
    _, rstd, y = ref.norm(x, w, EPS, r)
    g = group or d
    n = -(-d // g)
    assert got.y.shape == (rows, d) and got.scales.shape == (rows, n)
    pad = torch.nn.functional.pad(y, (0, n * g - d)).view(rows, n, g)
    scale = pad.abs().amax(2) / 448.0
    err = ((chain(d) + 8) * U32 * y.abs()
           + (x.double().abs() + r.double().abs()) * U32 * rstd[:, None] * w.double().abs())
    eg = torch.nn.functional.pad(err, (0, n * g - d)).view(rows, n, g).amax(2) / 448.0
    assert ((got.scales.double() - scale).abs() <= eg + 2 * U32 * scale).all()
    wide = got.scales.double().repeat_interleave(g, 1)[:, :d]
    back = got.y.double() * wide
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 of the scale below 2^-6
    step = torch.maximum(y.abs() * 2.0 ** -4, wide * 2.0 ** -10)
    assert ((back - y).abs() <= step * 1.001 + err + 4 * U32 * y.abs()).all()
    # the largest of every group takes the largest code
    codes = torch.nn.functional.pad(got.y.float(), (0, n * g - d)).view(rows, n, g)
    assert (codes.abs().amax(2) == 448.0).all()


def test_8bit_zeros_and_tiny_groups(dev):
    x = torch.zeros(3, 256, device=dev)
    x[1, :128] = 1.0
    x[2] = 1e-38
    w = torch.ones(256, device=dev)
    got = det.det_rms_norm(x, w, eps=1.0, quant=E4M3, group=128)
    tiny = 2.0 ** -100 / 448.0
    assert (got.y[0].float() == 0).all() and (got.scales[0] == tiny).all()
    assert (got.y[1, 128:].float() == 0).all() and got.scales[1, 1] == tiny
    assert (got.y[1, :128].float() == 448).all() and (got.y[2].float() == 0).all()


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_non_finite_rows_stay_alone(dev, t):
    x, r, w = inputs(6, 700, t, dev, 5)
    clean = det.det_rms_norm(x, w, residual=r)
    x[1, 3], x[4, 699] = float("nan"), float("inf")
    got = det.det_rms_norm(x, w, residual=r)
    for i in (0, 2, 3, 5):
        assert same_bits(got.y[i], clean.y[i])
    assert got.y[1].isnan().all()
    assert got.y[4, 699].isnan() and (got.y[4, :699] == 0).all()
    q = det.det_rms_norm(x, w, residual=r, quant=E4M3, group=64)
    assert q.y[1].float().isnan().all() and q.scales[1].isnan().all()
    assert not q.y[0].float().isnan().any()


def test_zero_rows_and_leading_dimensions(dev):
    w = torch.ones(96, device=dev)
    for shape in ((0, 96), (2, 0, 96)):
        got = det.det_rms_norm(torch.empty(shape, device=dev), w)
        assert got.y.shape == shape and got.rstd.shape == shape[:-1]
        dx, dw = det.det_rms_norm_backward(got.y, got.y, w, got.rstd)
        assert dx.shape == shape and (dw == 0).all()
    x, r, w = inputs(12, 96, torch.bfloat16, dev, 3)
    flat = det.det_rms_norm(x, w, residual=r)
    deep = det.det_rms_norm(x.view(3, 4, 96), w, residual=r.view(3, 4, 96))
    assert deep.y.shape == (3, 4, 96) and same_bits(deep.y.view(12, 96), flat.y)
    one = det.det_rms_norm(x[0], w, residual=r[0])
    assert one.rstd.shape == () and same_bits(one.y, flat.y[0])


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("d", [96, 1000, 4096, 9000])
def test_rows_views_and_places_keep_their_bits(dev, d, t):
    x, r, w = inputs(37, d, t, dev, d)
    want = det.det_rms_norm(x, w, residual=r, quant=E4M3, group=32)
    again = det.det_rms_norm(x, w, residual=r, quant=E4M3, group=32)
    alone = det.det_rms_norm(x[11:12], w, residual=r[11:12], quant=E4M3, group=32)
    for a, b, c in zip(want, again, alone):
        assert same_bits(a, b) and same_bits(a[11:12], c)
    # rows of a wider buffer, one element past an aligned start
    wide = torch.full((37, d + 9), float("nan"), device=dev).to(t)
    wide[:, 1:d + 1] = x
    shifted = torch.full((d + 1,), 0.0, device=dev).to(t)
    shifted[1:] = w
    for a, b in zip(want, det.det_rms_norm(wide[:, 1:d + 1], shifted[1:], residual=r, quant=E4M3,
                                           group=32)):
        assert same_bits(a, b)
    # on another stream, its results waited for
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = det.det_rms_norm(x, w, residual=r, quant=E4M3, group=32)
    torch.cuda.current_stream().wait_stream(s)
    assert same_bits(other.y, want.y)


@pytest.mark.parametrize("d", [96, 4096, 20001])
def test_h_in_place_of_an_input(dev, d):
    t = torch.bfloat16
    x, r, w = inputs(5, d, t, dev, d)
    want = det.det_rms_norm(x, w, residual=r, quant=E4M3)
    for replaced in (0, 1):
        ins = [x.clone(), r.clone()]
        y = torch.empty(5, d, dtype=E4M3, device=dev)
        sc, rstd = torch.empty(5, device=dev), torch.empty(5, device=dev)
        st = det.lib().det_rms_norm(ins[0].data_ptr(), d, ins[1].data_ptr(), d, w.data_ptr(), 5, d,
                                    det.DET_BF16, 1e-6, ins[replaced].data_ptr(), y.data_ptr(),
                                    det.DET_E4M3, 0, sc.data_ptr(), rstd.data_ptr(),
                                    torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert same_bits(ins[replaced], want.h) and same_bits(y, want.y)
        assert same_bits(sc, want.scales[:, 0])


BACK = [(1, 1), (3, 7), (9, 64), (2, 512), (7, 513), (5, 2048), (6, 2049), (3, 4096), (5, 5001),
        (2, 8192), (3, 8193), (2, 16384), (9, 16390), (3000, 24), (2100, 520)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,d", BACK)
@pytest.mark.parametrize("stream", [False, True])
def test_norm_backward(dev, rows, d, t, stream):
    x, r, w = inputs(rows, d, t, dev, d + rows)
    f = det.det_rms_norm(x, w, residual=r)
    dy = randn((rows, d), t, dev, 77, 1e-2)
    dh = randn((rows, d), t, dev, 78, 1e-2) if stream else None
    dx, dw = det.det_rms_norm_backward(dy, f.h, w, f.rstd, dh)
    want, dwant = ref.norm_backward(dy, f.h, w, f.rstd, dh)
    rs = f.rstd.double()[:, None]
    xhat = f.h.double() * rs
    g = (dy.double() * w.double()).abs()
    # the row's sum: a chain of (chain + 4) roundings of terms of these magnitudes
    terms = rs * (g + xhat.abs() * (g * xhat.abs()).mean(1, keepdim=True))
    bound = (chain(d) + 12) * U32 * terms + half(t) * want.abs() * 1.001 + floor_of(t)
    if stream:
        bound += 2 * U32 * dh.double().abs()
    assert ((dx.double() - want).abs() <= bound).all()
    # the rows' sum: a strip of at most 8 rows here, the strips of a workgroup and of a lane, the
    # levels above
    depth = 8 + -(-rows // 64) + 6 + 4
    mags = (dy.double() * xhat).abs().sum(0)
    assert ((dw.double() - dwant).abs()
            <= depth * U32 * mags + half(t) * dwant.abs() * 1.001 + floor_of(t)).all()
    again = det.det_rms_norm_backward(dy, f.h, w, f.rstd, dh)
    assert same_bits(again[0], dx) and same_bits(again[1], dw)
    i = rows // 2
    alone = det.det_rms_norm_backward(dy[i:i + 1], f.h[i:i + 1], w, f.rstd[i:i + 1],
                                      None if dh is None else dh[i:i + 1])
    assert same_bits(alone[0], dx[i:i + 1])


def test_norm_backward_strided_and_in_place(dev):
    t, rows, d = torch.float16, 11, 777
    x, r, w = inputs(rows, d, t, dev, 9)
    f = det.det_rms_norm(x, w, residual=r)
    dy, dh = randn((rows, d), t, dev, 1, 1e-2), randn((rows, d), t, dev, 2, 1e-2)
    want = det.det_rms_norm_backward(dy, f.h, w, f.rstd, dh)
    wide = torch.zeros(3, rows, d + 5, dtype=t, device=dev)
    for i, v in enumerate((dy, f.h, dh)):
        wide[i, :, 3:3 + d] = v
    got = det.det_rms_norm_backward(wide[0, :, 3:3 + d], wide[1, :, 3:3 + d], w, f.rstd,
                                    wide[2, :, 3:3 + d])
    assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
    for i in range(3):
        ins = [dy.clone(), f.h.clone(), dh.clone()]
        dw = torch.empty_like(w)
        ws = torch.empty(det.det_rms_norm_backward_workspace_size(rows, d, det.DET_F16),
                         dtype=torch.uint8, device=dev)
        assert det.lib().det_rms_norm_backward(
            ins[0].data_ptr(), d, ins[1].data_ptr(), d, w.data_ptr(), f.rstd.data_ptr(),
            ins[2].data_ptr(), d, rows, d, det.DET_F16, ins[i].data_ptr(), dw.data_ptr(),
            ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
        assert same_bits(ins[i], want[0]) and same_bits(dw, want[1])


@pytest.mark.parametrize("d", [5, 300, 2100])
def test_gradient_against_differences(dev, d):
    rows = 4
    x, r, w = inputs(rows, d, torch.float32, dev, 21)
    for v in (x, r, w):
        v.requires_grad_(True)
    y, h = det.rms_norm(x, w, r)
    cy, ch = randn((rows, d), torch.float32, dev, 22), randn((rows, d), torch.float32, dev, 23)
    ((y * cy).sum() + (h * ch).sum()).backward()

    def value(a, b, c):
        hh, _, yy = ref.norm(a, c, EPS, b)
        return float((yy * cy.double()).sum() + (hh * ch.double()).sum())

    args = [v.detach().double() for v in (x, r, w)]
    for n, v in enumerate((x, r, w)):
        step = randn(v.shape, torch.float32, dev, 30 + n).double()
        lo, hi = list(args), list(args)
        e = 1e-5
        lo[n], hi[n] = args[n] - e * step, args[n] + e * step
        slope = (value(*hi) - value(*lo)) / (2 * e)
        got = float((v.grad.double() * step).sum())
        # differences: third derivatives times e^2 and the values' rounding over e, 64 bits
        size = float((v.grad.double() * step).abs().sum())
        assert abs(got - slope) <= 1e-5 * size + 1e-6, (n, got, slope)


def test_norm_autograd_paths(dev):
    x, r, w = inputs(6, 130, torch.bfloat16, dev, 50)
    f = det.det_rms_norm(x, w)
    dy = randn((6, 130), torch.bfloat16, dev, 51)
    want = det.det_rms_norm_backward(dy, x, w, f.rstd)
    a, b = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    det.rms_norm(a, b).backward(dy)
    assert same_bits(a.grad, want[0]) and same_bits(b.grad, want[1])
    # only h is used further: the norm's own part is zero
    a, c = x.clone().requires_grad_(True), r.clone().requires_grad_(True)
    _, h = det.rms_norm(a, w, c)
    h.backward(dy)
    assert torch.equal(a.grad, dy) and torch.equal(c.grad, dy)
    # a broadcast gradient
    a = x.clone().requires_grad_(True)
    det.rms_norm(a, w).sum().backward()
    one = det.det_rms_norm_backward(torch.ones_like(x), x, w, f.rstd)
    assert same_bits(a.grad, one[0])
