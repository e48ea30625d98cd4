"""The recurrent model's operators where a shortcut, a grid's bound or a sum's order could show: gates
that are not finite beside a state of zero, more tiles than a grid holds, factors whose parts err to
one side, long sums of a few rows' logits, tokens by the ten thousand of a small vocabulary."""
import pytest
import torch

from lm_reference import IDS, TYPES, randn
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu


def steps_of(gate, x, state, sigmoid):
    """The recurrence one step after the other in 64 bits; NaN and infinity as they come."""
    a = gate.double().sigmoid() if sigmoid else gate.double()
    b = gate.double().neg().sigmoid() * x.double() if sigmoid else x.double()
    h, out = torch.zeros_like(a[:, 0]) if state is None else state.double(), []
    for t in range(a.shape[1]):
        h = a[:, t] * h + b[:, t]
        out.append(h)
    return torch.stack(out, 1)


# one workgroup a sequence, and several
@pytest.mark.parametrize("steps", [20, 300, 1300])
@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_gate_that_is_not_finite_shows_from_its_step_on(dev, t, steps, bad):
    """At the first step of a sequence, of a span (8 steps) and of a chunk (128), at others, beside a
    state of zero: whole numbers, so that the values before it are exact."""
    at = [s for s in (0, 8, 3, 128, 127, 136, 1024, 1031, steps - 1) if s < steps]
    gate, x = torch.ones(2, steps, 70, device=dev, dtype=t), torch.zeros(2, steps, 70, device=dev, dtype=t)
    for c, s in enumerate(at):
        gate[:, s, c] = bad      # every state before it is 0, and 0 * bad is NaN
    x[1, :, 20:] = 1
    for sigmoid in (False, True) if bad != bad else (False,):
        want = steps_of(gate, x, None, sigmoid)
        assert all(want[:, s:, c].isnan().all() for c, s in enumerate(at))
        for state in (None, torch.zeros(2, 70, device=dev)):
            got = det.det_gated_scan(gate, x, state, sigmoid)
            assert torch.equal(got.h.isnan(), want.isnan())
            assert torch.equal(got.state.isnan(), want[:, -1].isnan())
            if not sigmoid and t == torch.float32:
                assert torch.equal(got.h.nan_to_num(-1.0).double(), want.nan_to_num(-1.0))


@pytest.mark.parametrize("steps", [20, 300, 1300])
def test_gates_above_one_leave_a_state_of_zero(dev, steps):
    """Products of finite gates that overflow are no gates: a state of 0 stays 0, a bias adds up behind it."""
    gate, x = torch.full((1, steps, 70), 3e38, device=dev), torch.zeros(1, steps, 70, device=dev)
    got = det.det_gated_scan(gate, x)
    assert (got.h == 0).all() and (got.state == 0).all()
    gate[:, -1], x[:, -1] = 0.5, 3.0
    got = det.det_gated_scan(gate, x)
    assert (got.h[:, :-1] == 0).all() and (got.state == 3).all()


@pytest.mark.parametrize("steps", [8, 20, 300, 1300])
def test_negative_zeros_add_to_a_state_of_zero(dev, steps):
    """a * 0 + -0 is 0 for a gate that is not negative, however many steps a call has."""
    gate = torch.full((1, steps, 70), 0.5, device=dev)
    x = torch.full((1, steps, 70), -0.0, device=dev)
    got = det.det_gated_scan(gate, x)
    assert not torch.signbit(got.h).any() and not torch.signbit(got.state).any()


@pytest.mark.parametrize("batch", [4194297, (1 << 22) + 5])
def test_more_tiles_than_a_grid_of_whole_workgroups_holds(dev, batch):
    """Two channels a sequence take workgroups of 1024 threads, of which 4194303 fit into a grid and
    4194304, the next multiple of 8, do not.  Whole numbers, so that every sum is exact."""
    steps, d = 9, 2
    g = torch.Generator(dev).manual_seed(3)
    gate = torch.randint(0, 2, (batch, steps, d), generator=g, device=dev, dtype=torch.int8)
    x = torch.randint(-3, 4, (batch, steps, d), generator=g, device=dev, dtype=torch.int8)
    state = torch.randint(-6, 7, (batch, d), generator=g, device=dev, dtype=torch.int8)
    h, now = torch.empty_like(x), state
    for i in range(steps):
        now = gate[:, i] * now + x[:, i]
        h[:, i] = now
    got = det.det_gated_scan(gate.half(), x.half(), state.float())
    assert torch.equal(got.h, h.half()) and torch.equal(got.state, now.float())
    dgate, dx, first = det.det_gated_scan_backward(x.half(), gate.half(), x.half(), got.h, state.float(),
                                                   state.float())
    e, before = state, torch.cat([state[:, None], h[:, :-1]], 1)
    for i in reversed(range(steps)):
        e = x[:, i] + e      # G of the step
        assert torch.equal(dx[:, i], e.half())
        assert torch.equal(dgate[:, i], (e.short() * before[:, i]).half())
        e = gate[:, i] * e
    assert torch.equal(first, e.float())


@pytest.mark.parametrize("rows", [64, 100])      # tiles of 32 columns, and of 128
def test_f32_products_are_off_to_either_side(dev, rows):
    """One entry and a width of one: lse is the product x w itself.  Of the parts of a factor the second is
    at most 2^-7 of it and the third 2^-16, so the three products left out are at most (1 + 2^-9) 2^-22 of x
    w; the five smaller sums are at most 2^-5 of it, each off by a step 2^-23 of that; the last addition
    rounds by 2^-24.  In all below 2.7 * 2^-23.

    The mean over many w: w's third part, either sign alike, times the mean of x's second, 2^-8, has a
    standard deviation of 2^-24 / sqrt(3) a w; all else differs from row to row."""
    at = torch.zeros(rows, dtype=torch.int64, device=dev)
    special = torch.tensor([1 + 2.0 ** -7 - 2.0 ** -23, 2 - 2.0 ** -23, 1 + 2.0 ** -8, 1.0], device=dev)
    errors, seeds = [], 256
    for seed in range(seeds):
        g = torch.Generator(dev).manual_seed(seed)
        x, w = 1 + torch.rand(rows, 1, generator=g, device=dev), 1 + torch.rand(1, 1, generator=g, device=dev)
        x[:4, 0] = special
        for one in (w, special[seed % 4].view(1, 1)):
            got = det.det_linear_cross_entropy(x, one, at)
            want = (x.double() * one.double())[:, 0]
            rel = (got.lse.double() - want) / want
            assert rel.abs().max() <= 2.7 * 2.0 ** -23, float(rel.abs().max()) * 2 ** 23
            assert (got.loss == 0).all()
            if one is w:
                errors.append(rel[4:])
    errors = torch.cat(errors)
    allowed = 2.0 ** -24 / (3 * seeds) ** 0.5 + 2.7 * 2.0 ** -23 / errors.numel() ** 0.5
    assert errors.mean().abs() <= 4 * allowed


@pytest.mark.parametrize("rows", [5, 100])
def test_f32_entries_masked_by_the_lowest_float(dev, rows):
    """Entries whose weight is the type's lowest value have a logit as low, or -infinity, and take no part;
    a NaN still reaches its row alone."""
    d = 40
    x = 0.5 + randn((rows, d), torch.float32, dev, 1).abs()
    w = randn((300, d), torch.float32, dev, 2, 0.1)
    at = torch.arange(rows, device=dev) % 200
    kept = det.det_linear_cross_entropy(x, w[:200].contiguous(), at)
    w[200:] = torch.finfo(torch.float32).min
    got = det.det_linear_cross_entropy(x, w, at)
    # the same logits in other tiles: the sums' order, at most 300 terms
    assert ((got.lse - kept.lse).abs() <= 300 * 2.0 ** -24 * (1 + kept.lse.abs())).all()
    one = torch.zeros(300, d, device=dev)
    one[200:, 3] = torch.finfo(torch.float32).min
    got = det.det_linear_cross_entropy(x, one, at)      # finite, or -infinity where x is above 1
    assert ((got.lse.double() - torch.log(torch.tensor(200.0).double())).abs() <= 1e-5).all()
    x[2, 7] = float("nan")
    got = det.det_linear_cross_entropy(x, w, at)
    assert torch.equal(got.lse.isnan(), torch.arange(rows, device=dev) == 2)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,d", [(1, 4096), (64, 4096), (3, 1000), (5, 4095)])
def test_long_sums_of_few_rows_go_through_several_accumulators(dev, rows, d, t):
    """A logit of 1024 in its first product, behind it products that add half a step 2^-13 of it every 16: an
    accumulator that holds the 1024 loses them.  Four take the steps in turn (f32: two), so that one loses a
    quarter (half), each at most half a step, and the joins round three times.  One entry: lse is the logit."""
    x, w = torch.ones(rows, d, device=dev), torch.full((1, d), 2.0 ** -18, device=dev)
    w[0, 0] = 1024.0
    got = det.det_linear_cross_entropy(x.to(t), w.to(t), torch.zeros(rows, dtype=torch.int64, device=dev))
    want = 1024 + (d - 1) * 2.0 ** -18
    steps = -(-d // 16) // (2 if t == torch.float32 else 4)
    assert ((got.lse.double() - want).abs() <= (steps + 4) * 2.0 ** -14).all()


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_sequences_keep_their_bits_across_the_widths_of_a_tile(dev, t):
    """128 tiles of 64 words and one more: halved tiles, then whole ones, and a sequence alone."""
    steps, d = 140, 128 if t != torch.float32 else 64      # a tile a sequence
    gate, x = randn((129, steps, d), t, dev, 1), randn((129, steps, d), t, dev, 2)
    dh = randn((129, steps, d), t, dev, 3)
    outs = []
    for n in (129, 128, 1):
        r = det.det_gated_scan(gate[:n], x[:n], None, True)
        outs.append([*r, *det.det_gated_scan_backward(dh[:n], gate[:n], x[:n], r.h, None, None, True)[:2]])
    for more in outs[:2]:
        for a, b in zip(more, outs[2]):
            assert torch.equal(a[:1], b)
    for a, b in zip(outs[0], outs[1]):
        assert torch.equal(a[:128], b)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,vocab", [(65537, 1), (70000, 2), (65537, 256), (70001, 257), (66000, 100000)])
def test_table_gradients_of_many_tokens_and_few_or_no_entries(dev, n, vocab, dtype):
    """Through the radix sort: a vocabulary of one entry, around a digit's 256, and tokens of which none
    counts.  Whole numbers below 2^24, so that every sum is exact."""
    g = torch.Generator(dev).manual_seed(n)
    ids = torch.randint(-1, vocab + 1, (n,), generator=g, device=dev).to(dtype)
    dout = torch.randint(-3, 4, (n, 9), generator=g, device=dev).float()
    got = det.det_embedding_backward(dout, ids, vocab)
    on = (ids >= 0) & (ids < vocab)
    want = torch.zeros(vocab + 1, 9, dtype=torch.float64, device=dev)
    want.index_add_(0, torch.where(on, ids, vocab).long(), dout.double())
    assert torch.equal(got.double(), want[:-1])
    none = torch.where(on, torch.full_like(ids, vocab), ids)
    assert (det.det_embedding_backward(torch.full_like(dout, float("nan")), none, vocab) == 0).all()
