"""det_relative_bias and its table's gradient on the GPU against 64-bit statements whose buckets
are found in whole numbers.  Without scores the output is the table's own values, bit for bit;
with them one f32 addition and the type's rounding; the table's gradient sums in f32 along at most
128 rows and 512 diagonals in 8 steps and 6 levels (in fact along 8 rows), and the rest in f64."""
import math

import pytest
import torch

import lm_reference as ref
from lm_reference import IDS, TYPES, U32, floor_of, half, randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


CASES = [  # batch, heads, q, k, buckets, distance, two_sided, causal, offsets, lengths
    (1, 1, 1, 1, 32, 128, True, False, 0, None),
    (1, 3, 5, 9, 32, 128, True, False, 0, None),
    (2, 2, 1, 65, 32, 128, False, True, [64, 12], [65, 13]),
    (3, 4, 33, 70, 16, 64, False, True, 37, [70, 41, 1]),
    (2, 1, 130, 130, 64, 1024, True, True, 0, [130, 77]),
    (1, 2, 200, 2050, 32, 100, True, False, 1850, None),
    (2, 5, 77, 515, 32, 500, False, False, -3, [0, -4]),
    (2, 2, 300, 64, 7, 20, False, True, -100, [64, 20]),
    (1, 1, 513, 1030, 9, 33, True, True, 200, None),
    (2, 3, 64, 4097, 32, 128, False, False, [4033, 0], [4097, 9000]),
    (1, 2, 1000, 8, 4, 5, True, False, 500, None),
]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_bias_and_gradient(dev, case, t):
    b, h, q, k, buckets, distance, two, causal, off, lens = case
    maps = ref.bias_maps(b, q, k, buckets, distance, two, causal, off, lens, dev)
    how = dict(max_distance=distance, bidirectional=two, causal=causal,
               q_offset=off if isinstance(off, int) else i32(off, dev),
               lengths=None if lens is None else i32(lens, dev))
    table = randn((buckets, h), t, dev, 1)
    got = det.det_relative_bias(table, q, k, **how)
    nb = b if lens is not None or not isinstance(off, int) else 1
    want = ref.bias(table, maps)[:nb]
    assert got.shape == want.shape and torch.equal(got.double(), want)
    # scores, NaN and infinities in the masked places among them
    scores = randn((b, h, q, k), t, dev, 2, 2.0)
    left = maps[1][:, None].expand_as(scores)
    for junk in (float("nan"), float("inf"), float("-inf"), torch.finfo(t).min):
        dirty = torch.where(left, scores, junk)
        got = det.det_relative_bias(table, q, k, scores=dirty, **how)
        want = ref.bias(table, maps, scores)
        size = torch.where(left, want.abs(), 0.0)
        err = torch.where(left, (got.double() - want).abs(), 0.0)
        assert (err <= size * (half(t) + 2 * U32) + floor_of(t)).all()
        assert (got[~left] == -math.inf).all()
    # in place
    buf = scores.clone()
    assert det.det_relative_bias(table, q, k, scores=buf, out=buf, **how) is buf
    assert same_bits(buf, det.det_relative_bias(table, q, k, scores=scores, **how))

    dout = randn((b, h, q, k), t, dev, 3, 1e-2)
    dwant, sizes, dscores = ref.bias_backward(dout, maps, buckets)
    bound = (128 + 8 + 6 + 2) * U32 * sizes + half(t) * dwant.abs() * 1.001 + floor_of(t)
    dirty = torch.where(left, dout, float("nan"))
    ds = torch.full_like(dout, 5.0)
    got = det.det_relative_bias_backward(dirty, buckets, dscores=ds, **how)
    assert ((got.double() - dwant).abs() <= bound).all()
    assert torch.equal(ds.double(), dscores)
    assert same_bits(det.det_relative_bias_backward(dout, buckets, **how), got)


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("buckets,distance", [(32, 128), (32, 256), (16, 64), (64, 1024), (32, 100),
                                              (64, 500), (5, 3), (30, 2000), (128, 4000)])
def test_every_distance_falls_into_its_bucket(dev, buckets, distance, two):
    if (buckets // 2 if two else buckets) // 2 >= distance:
        pytest.skip("no room beyond the near buckets")
    n = distance + 300
    table = torch.arange(buckets, device=dev, dtype=torch.float32)[:, None].contiguous()
    got = det.det_relative_bias(table, 1, 2 * n + 1, max_distance=distance, bidirectional=two,
                                q_offset=n)
    want = [ref.bucket(r, buckets, distance, two) for r in range(-n, n + 1)]
    assert got[0, 0, 0].tolist() == want


def test_far_offsets(dev):
    # the positions of a long cache: only the distance counts
    table = randn((32, 2), torch.bfloat16, dev, 4)
    near = det.det_relative_bias(table, 3, 100, q_offset=97)
    assert torch.equal(det.det_relative_bias(table, 3, 100, q_offset=1 << 35)[0, 1],
                       table[15, 1].expand(3, 100))
    assert torch.equal(det.det_relative_bias(table, 3, 100, q_offset=-(1 << 35))[0, 0],
                       table[31, 0].expand(3, 100))
    big = i32([97, (1 << 31) - 1], dev)
    got = det.det_relative_bias(table, 3, 100, q_offset=big)
    assert torch.equal(got[0], near[0])
    assert torch.equal(got[1, 0], table[15, 0].expand(3, 100))


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_strides_and_views(dev, t):
    b, h, q, k = 2, 3, 40, 211
    table = randn((32, h), t, dev, 5)
    lens = i32([211, 100], dev)
    base = randn((q, b, h, k + 6), t, dev, 6)
    view = base[..., 1:k + 1].permute(1, 2, 0, 3)          # rows contiguous, the rest strided
    want = det.det_relative_bias(table, q, k, scores=view.contiguous(), causal=True, q_offset=171,
                                 lengths=lens)
    assert same_bits(det.det_relative_bias(table, q, k, scores=view, causal=True, q_offset=171,
                                           lengths=lens), want)
    shared = view[:1, :1].expand(b, h, q, k)               # one map of scores for all heads
    got = det.det_relative_bias(table, q, k, scores=shared)
    assert same_bits(got, det.det_relative_bias(table, q, k, scores=shared.contiguous()))
    for v in (view, shared):
        d = det.det_relative_bias_backward(v, 32, lengths=lens)
        assert same_bits(d, det.det_relative_bias_backward(v.contiguous(), 32, lengths=lens))
    one = det.det_relative_bias_backward(view, 32)
    for _ in range(3):
        assert same_bits(det.det_relative_bias_backward(view, 32), one)


def test_empty(dev):
    table = torch.ones(32, 4, device=dev)
    for b, q, k in ((0, 3, 5), (2, 0, 5), (2, 3, 0)):
        s = torch.empty(b, 4, q, k, device=dev)
        assert det.det_relative_bias(table, q, k, scores=s).shape == (b, 4, q, k)
        d = det.det_relative_bias_backward(s, 32)
        assert d.shape == (32, 4) and (d == 0).all()


@pytest.mark.parametrize("causal,ragged", [(False, False), (True, False), (False, True)])
def test_gradient_against_differences(dev, causal, ragged):
    b, h, q, k, buckets = 2, 2, 9, 14, 8
    lens = [14, 6] if ragged else None
    maps = ref.bias_maps(b, q, k, buckets, 10, True, causal, 5, lens, dev)
    table = randn((buckets, h), torch.float32, dev, 7).requires_grad_(True)
    scores = randn((b, h, q, k), torch.float32, dev, 8).requires_grad_(True)
    c = randn((b, h, q, k), torch.float32, dev, 9)
    out = det.relative_bias(table, q, k, scores, max_distance=10, causal=causal, q_offset=5,
                            lengths=None if lens is None else i32(lens, dev))
    # what attention does with it: a softmax whose rows without a key give nothing
    p = torch.nan_to_num(out.softmax(-1))
    (p * c).sum().backward()

    def value(tb, sc):
        o = ref.bias(tb, maps, sc)
        return float((torch.nan_to_num(o.softmax(-1)) * c.double()).sum())

    a = [table.detach().double(), scores.detach().double()]
    for n, v in enumerate((table, scores)):
        grad = torch.nan_to_num(v.grad.double())
        step = randn(v.shape, torch.float32, dev, 40 + n).double()
        e = 1e-5
        lo, hi = list(a), list(a)
        lo[n], hi[n] = a[n] - e * step, a[n] + e * step
        slope = (value(*hi) - value(*lo)) / (2 * e)
        got = float((grad * step).sum())
        assert abs(got - slope) <= 1e-5 * float((grad * step).abs().sum()) + 1e-6
