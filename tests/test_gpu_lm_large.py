"""The language-model operators at the sizes that choose other kernels than small calls do: inputs
of 128 MiB and more (loaded past the caches), strips and walks longer than the shortest, and more
rows, heads and tiles than one launch starts workgroups for.  What a row's bits may not depend on is
compared bit for bit with smaller calls; sums over rows are compared with 64 bits.

Tolerances: U = 2^-24.  A strip's chain is at most rows / 256 long (4 where that is less), 3 more
teams of a workgroup, 2048 / 256 strips a lane, 8 levels of the tree; a term dy * (h * rstd) is off by
2 U.  The table's gradient adds 8 rows in float (7 roundings) and the rest in double."""
import math

import pytest
import torch

import lm_reference as ref
from lm_reference import IDS, TYPES, U32, floor_of, half, randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
PAST = 1 << 27          # bytes of input from which on the loads go past the caches


def size(t):
    return torch.finfo(t).bits // 8


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ norm

WIDTHS = [200, 777, 1500, 4001, 5001, 8001, 12345]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("residual,group", [(False, None), (True, None), (False, 0), (True, 128)])
def test_norm_past_the_caches(dev, d, t, residual, group):
    each = d * size(t) * (2 if residual else 1)
    rows = PAST // each + 7
    x, w = randn((rows, d), t, dev, d), randn((d,), t, dev, 1)
    r = randn((rows, d), t, dev, d + 2) if residual else None
    how = {"quant": E4M3, "group": group} if group is not None else {}
    got = det.det_rms_norm(x, w, residual=r, **how)
    assert rows * each >= PAST
    for i in range(0, rows, rows // 3):
        part = det.det_rms_norm(x[i:i + rows // 3], w,
                                residual=None if r is None else r[i:i + rows // 3], **how)
        for a, b in zip(got, part):
            assert (a is None and b is None) or same_bits(a[i:i + rows // 3], b)


@pytest.mark.parametrize("rows,d", [(8500000, 8), (1031 * 2035, 1032)])
def test_norm_of_more_rows_than_workgroups(dev, rows, d):
    """4 rows a workgroup and one: the second row of a workgroup finds the first one's LDS."""
    t, period = torch.bfloat16, 1031 if d > 1000 else 8500
    x, w = randn((period, d), t, dev, 3), randn((d,), t, dev, 4)
    for how in ({}, {"quant": E4M3}):
        want = det.det_rms_norm(x, w, **how)
        got = det.det_rms_norm(x.repeat(rows // period, 1), w, **how)
        for i in (0, 2, 3):
            if want[i] is not None:
                a = got[i].view(torch.uint8).view(rows // period, -1)
                assert (a == want[i].reshape(-1).view(torch.uint8)).all()


def test_norm_of_more_long_rows_than_workgroups(dev):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GiB of free GPU memory")
    t, period, d = torch.bfloat16, 1024, 16385
    reps = (1 << 21) // period + 1
    x, w = randn((period, d), t, dev, 3), randn((d,), t, dev, 4)
    want = det.det_rms_norm(x, w, quant=E4M3)
    wide = x.repeat(reps, 1)
    got = det.det_rms_norm(wide, w, quant=E4M3)
    for i in range(reps):
        at = slice(i * period, (i + 1) * period)
        for j in (0, 2, 3):
            assert same_bits(got[j][at], want[j])
    del wide, got
    torch.cuda.empty_cache()


def check_backward(rows, d, t, dev, dh):
    h, dy = randn((rows, d), t, dev, 5), randn((rows, d), t, dev, 6, 1e-2)
    w, extra = randn((d,), t, dev, 7), randn((rows, d), t, dev, 8, 1e-2) if dh else None
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dx, dw = det.det_rms_norm_backward(dy, h, w, rstd, extra)
    for i in range(0, rows, rows // 3):
        at = slice(i, i + rows // 3)
        part, _ = det.det_rms_norm_backward(dy[at], h[at], w, rstd[at], None if extra is None else extra[at])
        assert same_bits(dx[at], part)
    dwant = torch.zeros(d, dtype=torch.float64, device=dev)
    sizes = torch.zeros_like(dwant)
    for i in range(0, rows, 1 + (1 << 25) // d):
        at = slice(i, i + 1 + (1 << 25) // d)
        terms = dy[at].double() * (h[at].double() * rstd[at].double()[:, None])
        dwant += terms.sum(0)
        sizes += terms.abs().sum(0)
    depth = max(4, -(-rows // 256)) + 3 + 8 + 8 + 2
    assert ((dw.double() - dwant).abs()
            <= depth * U32 * sizes + half(t) * dwant.abs() * 1.001 + floor_of(t)).all()
    again = det.det_rms_norm_backward(dy, h, w, rstd, extra)
    assert same_bits(again[0], dx) and same_bits(again[1], dw)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dh", [False, True])
def test_norm_backward_past_the_caches(dev, d, t, dh):
    check_backward(PAST // (d * size(t) * (3 if dh else 2)) + 7, d, t, dev, dh)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,d", [(20011, 96), (40000, 24), (9001, 600), (9000, 1500), (3001, 2500),
                                    (1500, 4100), (1100, 9000), (1030, 16390)])
def test_norm_backward_of_long_strips(dev, rows, d, t):
    check_backward(rows, d, t, dev, rows % 2 == 1)


# ------------------------------------------------------------------ relative position bias

def line_of(buckets, distance, two_sided, dev):
    """Buckets of the relative positions -distance .. distance; those beyond are like the ends."""
    return torch.tensor([ref.bucket(r, buckets, distance, two_sided)
                         for r in range(-distance, distance + 1)], device=dev)


def places(q, k, line, causal, off, length, dev):
    """(bucket, unmasked), [q, k], of one sequence"""
    far = (line.numel() - 1) // 2
    i, j = torch.arange(q, device=dev)[:, None] + off, torch.arange(k, device=dev)[None]
    left = torch.ones(q, k, dtype=torch.bool, device=dev)
    if causal:
        left &= j <= i
    if length is not None:
        left &= (j < length) & (i < length)
    return line[(j - i).clamp(-far, far) + far], left


BIAS = [  # batch, heads, q, k, type, buckets, distance, two_sided, causal, offset(s), lengths
    (4, 16, 1100, 2000, torch.bfloat16, 32, 128, False, True, 900, [2000, 1500, 37, 1999]),
    (3, 8, 1500, 2100, torch.float32, 32, 128, True, False, 0, None),
    (5, 7, 1300, 1501, torch.float16, 64, 1024, True, True, [201, 0, -50, 201, 1400], None),
    (16, 16, 2100, 300, torch.float16, 16, 64, True, False, 0, [300 - 11 * i for i in range(16)]),
    (2, 8, 1000, 1500, torch.bfloat16, 32, 128, True, False, 500, None),
    (3, 5, 777, 1003, torch.float32, 32, 256, False, True, 226, [1003, 600, 501]),
    (1, 300, 130, 4100, torch.float32, 7, 20, False, False, 3970, [4000]),
]


@pytest.mark.parametrize("case", BIAS, ids=str)
def test_bias_of_long_walks(dev, case):
    b, h, q, k, t, buckets, distance, two, causal, off, lens = case
    how = dict(max_distance=distance, bidirectional=two, causal=causal,
               q_offset=off if isinstance(off, int) else i32(off, dev),
               lengths=None if lens is None else i32(lens, dev))
    line = line_of(buckets, distance, two, dev)
    maps = [places(q, k, line, causal, off if isinstance(off, int) else off[i],
                   None if lens is None else lens[i], dev) for i in range(b)]
    table = randn((buckets, h), t, dev, 1)
    alone = det.det_relative_bias(table, q, k, **how)
    for i in range(alone.shape[0]):
        bk, left = maps[i]
        for j in range(h):
            assert torch.equal(alone[i, j], torch.where(left, table[:, j][bk], -math.inf))
    del alone
    # one float addition and one rounding, whatever stands in the masked places
    scores = randn((b, h, q, k), t, dev, 2, 2.0)
    for i in range(b):
        scores[i].masked_fill_(~maps[i][1], math.nan)
    out = det.det_relative_bias(table, q, k, scores=scores, **how)
    for i in range(b):
        bk, left = maps[i]
        for j in range(h):
            want = (scores[i, j].float() + table[:, j].float()[bk]).to(t)
            assert torch.equal(out[i, j], torch.where(left, want, -math.inf))
    assert det.det_relative_bias(table, q, k, scores=scores, out=scores, **how) is scores
    assert same_bits(scores, out)
    del scores, out

    dout = randn((b, h, q, k), t, dev, 3, 1e-2)
    for i in range(b):
        dout[i].masked_fill_(~maps[i][1], math.nan)
    ds = torch.full_like(dout, 5.0)
    got = det.det_relative_bias_backward(dout, buckets, dscores=ds, **how)
    want = torch.zeros(buckets, h, dtype=torch.float64, device=dev)
    sizes = torch.zeros_like(want)
    for i in range(b):
        bk, left = maps[i]
        hot = [(bk == c).flatten().nonzero()[:, 0] for c in range(buckets)]
        for j in range(h):
            g = torch.where(left, dout[i, j], 0.0)
            assert torch.equal(ds[i, j], g)
            g = g.double().flatten()
            for c in range(buckets):
                terms = g[hot[c]]
                want[c, j] += terms.sum()
                sizes[c, j] += terms.abs().sum()
    bound = 8 * U32 * sizes + half(t) * want.abs() * 1.001 + floor_of(t)
    assert ((got.double() - want).abs() <= bound).all()
    for _ in range(2):
        assert same_bits(det.det_relative_bias_backward(dout, buckets, **how), got)


@pytest.mark.parametrize("shape", [(2, 3, 300, 400), (1, 2, 1, 5000), (3, 5, 777, 1003), (3, 8, 1500, 2100)])
@pytest.mark.parametrize("causal", [False, True])
def test_table_gradient_adds_in_64_bits(dev, shape, causal):
    """Whole numbers whose sums over 8 rows fit 24 bits and whose total does not: one rounding."""
    b, h, q, k = shape
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    whole = torch.randint(-(1 << 19), 1 << 20, shape, generator=g, device=dev) | 1
    got = det.det_relative_bias_backward(whole.float(), 32, causal=causal, q_offset=k - q)
    bk, left = places(q, k, line_of(32, 128, True, dev), causal, k - q, None, dev)
    for c in range(32):
        sums = (whole * (left & (bk == c))).sum((0, 2, 3))
        assert sums.abs().max() < 1 << 52
        assert torch.equal(got[c], sums.double().float())


def test_bias_of_more_tiles_than_workgroups(dev):
    t = torch.bfloat16
    # heads of all sequences past 65535
    line = line_of(32, 128, True, dev)
    table = randn((32, 30000), t, dev, 11)
    scores = randn((3, 30000, 9, 5), t, dev, 12)
    lens = [5, 2, 4]
    got = det.det_relative_bias(table, 9, 5, scores=scores, q_offset=-3, lengths=i32(lens, dev))
    for i in range(3):
        bk, left = places(9, 5, line, False, -3, lens[i], dev)
        want = (scores[i].float() + table.float().t()[:, bk]).to(t)
        assert torch.equal(got[i], torch.where(left, want, -math.inf))
    # query tiles past 65535: 2048 rows each
    q = 65535 * 2048 + 5000
    table = randn((32, 1), t, dev, 13)
    got = det.det_relative_bias(table, q, 3, q_offset=-q + 700)
    near = places(2000, 3, line, False, -1300, None, dev)[0]      # the last 2000 rows
    assert torch.equal(got[0, 0, -2000:], table[:, 0][near])
    # positions far below the keys: every relative position is large
    assert (got[0, 0, :-2000] == table[31, 0]).all()
    del got
    # single queries: 32 rows a workgroup, 65535 workgroups
    table = randn((32, 60000), t, dev, 14)
    lens = [9 - i % 10 for i in range(40)]
    at = [n - 1 for n in lens]
    got = det.det_relative_bias(table, 1, 9, q_offset=i32(at, dev), lengths=i32(lens, dev), causal=True)
    for i in range(40):
        bk, left = places(1, 9, line, True, at[i], lens[i], dev)
        assert torch.equal(got[i], torch.where(left, table.t()[:, bk], -math.inf))


def test_table_gradient_of_more_tiles_than_workgroups(dev):
    b, h, k = 75, 60001, 3                       # 4.5 million tiles, 2^22 workgroups
    dout = randn((b, h, 1, k), torch.bfloat16, dev, 15)
    got = det.det_relative_bias_backward(dout, 8, max_distance=9, q_offset=1)
    bk, _ = places(1, k, line_of(8, 9, True, dev), False, 1, None, dev)
    for c in range(8):
        terms = dout[:, :, 0][:, :, bk[0] == c].double()
        want, sizes = terms.sum((0, 2)), terms.abs().sum((0, 2))
        bound = 8 * U32 * sizes + half(dout.dtype) * want.abs() * 1.001 + floor_of(dout.dtype)
        assert ((got[c].double() - want).abs() <= bound).all()


# ------------------------------------------------------------------ token log probabilities

def logits_of(rows, vocab, t, dev):
    x = randn((rows, vocab), t, dev, 21, 2.5)
    at = torch.randint(-vocab // 8, vocab, (rows,), generator=torch.Generator().manual_seed(3)).to(dev)
    x[torch.arange(rows, device=dev), at.clamp_min(0)] += 6.0
    return x, at


def compare_with_parts(x, at, top, scale, part):
    rows, dev = x.shape[0], x.device
    got = det.det_token_logprobs(x, at, scale, top)
    dlp, den = randn((rows,), torch.float32, dev, 22), randn((rows,), torch.float32, dev, 23)
    grad = det.det_token_logprobs_backward(x, at, got.lse, dlp, got.entropy, den, scale)
    for i in range(0, rows, part):
        s = slice(i, i + part)
        want = det.det_token_logprobs(x[s], at[s], scale, top)
        for a, b in zip(got, want):
            assert (a is None and b is None) or same_bits(a[s].contiguous(), b)
        assert same_bits(grad[s], det.det_token_logprobs_backward(
            x[s], at[s], want.lse, dlp[s], want.entropy, den[s], scale))
    det.det_token_logprobs_backward(x, at, got.lse, dlp, got.entropy, den, scale, out=x)
    assert same_bits(x, grad)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,bytes_a_row", [(300, 460001), (513, 270001), (700, 200003), (20000, 7001),
                                              (1500, 131071)])
@pytest.mark.parametrize("top", [0, 5])
def test_logprobs_past_the_caches(dev, rows, bytes_a_row, t, top):
    vocab = bytes_a_row // size(t)
    assert rows * vocab * size(t) >= PAST
    x, at = logits_of(rows, vocab, t, dev)
    compare_with_parts(x, at, top, 1.0 if top else 0.8, min(rows // 3, 250))


def test_logprobs_of_more_rows_than_workgroups(dev):
    # 2^21 workgroups forward, 2^22 backward
    rows, vocab = (1 << 22) + 77, 5
    x, at = logits_of(rows, vocab, torch.bfloat16, dev)
    compare_with_parts(x, at, 3, 1.25, 1 << 20)
