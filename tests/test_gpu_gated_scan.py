"""det_gated_scan and its backward pass on the GPU against 64-bit loops, at the lengths where the
kernels change (8 steps a span, 128 a chunk, several workgroups a sequence), padded and empty
sequences, and what holds bit for bit.  The bounds run along with the loops (recurrent_reference)."""
import pytest
import torch

import recurrent_reference as ref
from lm_reference import IDS, TYPES, U32, floor_of, half, randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu


def inputs(batch, steps, d, t, dev, seed, sigmoid):
    gate = randn((batch, steps, d), torch.float32, dev, seed) + 1 + randn((d,), torch.float32, dev, seed + 1)
    gate = gate if sigmoid else gate.sigmoid() * torch.where(randn((d,), torch.float32, dev, 3) > 1.5, -1.0, 1.0)
    return gate.to(t), randn((batch, steps, d), t, dev, seed + 2), randn((batch, d), torch.float32, dev, seed + 3)


def lengths_of(batch, steps, dev):
    some = [steps, 0, steps - 1, steps // 2, 1, steps + 5, -3]
    return torch.tensor([some[i % 7] for i in range(batch)], dtype=torch.int32, device=dev)


def near(got, want, bound, t):
    # subnormals of the sigmoid and its products are lost below 2^-126
    allowed = U32 * bound * 1.001 + half(t) * (want.abs() + U32 * bound) * 1.001 + floor_of(t) + 2.0 ** -120
    return ((got.double() - want).abs() <= allowed).all()


SIZES = [(1, 1, 1), (3, 1, 7), (2, 2, 130), (2, 8, 65), (7, 9, 33), (2, 16, 64), (1, 127, 5), (2, 128, 129),
         (7, 129, 3), (1, 300, 200), (3, 511, 31), (1, 513, 64), (1, 2000, 70), (7, 700, 2)]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("batch,steps,d", SIZES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("ragged", [False, True])
def test_forward_and_backward(dev, batch, steps, d, t, sigmoid, ragged):
    gate, x, state = inputs(batch, steps, d, t, dev, steps + d, sigmoid)
    lens = lengths_of(batch, steps, dev) if ragged else None
    state = state if (batch + d) % 2 else None
    if ragged:      # what lies past a length is not used, whatever it is
        past = torch.arange(steps, device=dev) >= lens[:, None]
        gate[past], x[past] = float("nan"), float("inf")
        clean = torch.where(past[..., None], torch.zeros_like(gate), gate), torch.where(
            past[..., None], torch.zeros_like(x), x)
    else:
        clean = gate, x
    got = det.det_gated_scan(gate, x, state, sigmoid, lens)
    h, end, eh, ee = ref.scan(*clean, state, sigmoid, lens)
    assert near(got.h, h, eh, t) and near(got.state, end, ee, torch.float32)
    dh = randn((batch, steps, d), t, dev, 91)
    if ragged:
        dh[past] = float("nan")
    ds = randn((batch, d), torch.float32, dev, 92) if d % 3 else None
    back = det.det_gated_scan_backward(dh, gate, x, got.h, state, ds, sigmoid, lens)
    dclean = torch.where(past[..., None], torch.zeros_like(dh), dh) if ragged else dh
    dg, dx, first, eg, ex, ef = ref.scan_backward(dclean, *clean, got.h, state, ds, sigmoid, lens)
    assert near(back[0], dg, eg, t) and near(back[1], dx, ex, t)
    if state is None:
        assert back[2] is None
    else:
        assert near(back[2], first, ef, torch.float32)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("d", [40, 301])
def test_bits_do_not_depend_on_what_is_beside(dev, d, t, sigmoid):
    """A sequence alone, among many (one workgroup a sequence, or several), its channels alone, its
    first steps alone, cut in two at a chunk's border, repeated, on another stream."""
    steps = 1300
    gate, x, state = inputs(3, steps, d, t, dev, d, sigmoid)
    got = det.det_gated_scan(gate, x, state, sigmoid)
    again = det.det_gated_scan(gate, x, state, sigmoid)
    assert same_bits(got.h, again.h) and same_bits(got.state, again.state)
    many = [torch.cat([v] * 60).contiguous() for v in (gate, x, state)]      # 180 sequences
    big = det.det_gated_scan(*many, sigmoid)
    assert same_bits(big.h[:3], got.h) and same_bits(big.h[177:], got.h)
    assert same_bits(big.state[3:6], got.state)
    one = det.det_gated_scan(gate[1:2], x[1:2], state[1:2], sigmoid)
    assert same_bits(one.h, got.h[1:2]) and same_bits(one.state, got.state[1:2])
    part = det.det_gated_scan(gate[..., 7:20].contiguous(), x[..., 7:20].contiguous(),
                              state[:, 7:20].contiguous(), sigmoid)
    assert same_bits(part.h, got.h[..., 7:20].contiguous())
    for n in (1, 5, 8, 9, 128, 200, 640):
        head = det.det_gated_scan(gate[:, :n].contiguous(), x[:, :n].contiguous(), state, sigmoid)
        assert same_bits(head.h, got.h[:, :n].contiguous()), n
        lens = torch.full((3,), n, dtype=torch.int32, device=dev)
        cut = det.det_gated_scan(gate, x, state, sigmoid, lens)
        assert same_bits(cut.state, head.state) and same_bits(cut.h[:, :n].contiguous(), head.h)
        assert (cut.h[:, n:] == 0).all()
    dh = randn((3, steps, d), t, dev, 5)
    back = det.det_gated_scan_backward(dh, gate, x, got.h, state, state, sigmoid)
    wide = det.det_gated_scan_backward(torch.cat([dh] * 60), many[0], many[1], big.h, many[2], many[2], sigmoid)
    for a, b in zip(back, wide):
        assert same_bits(a, b[60:63])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = det.det_gated_scan(gate, x, state, sigmoid)
    torch.cuda.current_stream().wait_stream(s)
    assert same_bits(other.h, got.h)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_decoding_step_by_step(dev, t):
    """Single tokens from a state kept in place follow the whole sequence's recurrence: to the bit
    inside a span's 8 steps, then within the bounds."""
    gate, x, state = inputs(4, 40, 97, t, dev, 7, True)
    kept, hs = state.clone(), []
    for i in range(40):
        r = det.det_gated_scan(gate[:, i:i + 1].contiguous(), x[:, i:i + 1].contiguous(), kept, True,
                               state_out=kept)
        assert r.state is kept or r.state.data_ptr() == kept.data_ptr()
        hs.append(r.h)
    whole = det.det_gated_scan(gate, x, state, True)
    got = torch.cat(hs, 1)
    assert same_bits(got[:, :8].contiguous(), whole.h[:, :8].contiguous())
    h, end, eh, ee = ref.scan(gate, x, state, True)
    assert near(got, h, eh, t) and near(kept, end, ee, torch.float32)
    with pytest.raises(det.DetError):      # longer calls read it again
        det.det_gated_scan(gate, x, state, True, state_out=state)


def test_saturated_gates_and_non_finite_values(dev):
    steps, d = 300, 66
    gate, x, state = inputs(2, steps, d, torch.float32, dev, 3, True)
    gate[:, :, 0], gate[:, :, 1], gate[:, :, 2] = 200.0, -200.0, float("inf")
    gate[:, :, 3] = float("-inf")
    got = det.det_gated_scan(gate, x, state, True)
    for c in (0, 2):      # everything is kept
        assert torch.equal(got.h[:, :, c], state[:, c:c + 1].expand(2, steps))
    for c in (1, 3):      # nothing is
        assert torch.equal(got.h[:, :, c], x[:, :, c])
    clean = got.h.clone()
    x[1, 100, 7] = float("nan")
    got = det.det_gated_scan(gate, x, state, True)
    assert got.h[1, 100:, 7].isnan().all() and same_bits(got.h[1, :100], clean[1, :100])
    assert same_bits(got.h[0], clean[0]) and same_bits(got.h[1, :, 8:], clean[1, :, 8:])
    # linear gates of 0 start afresh, of 1 add up
    one = torch.ones(1, steps, 64, device=dev)
    up = det.det_gated_scan(one, one)
    assert torch.equal(up.h[0, :, 0], torch.arange(1, steps + 1, device=dev).float())
    one[:, 150] = 0.0
    again = det.det_gated_scan(one, torch.ones_like(one))
    assert again.h[0, 150, 3] == 1 and again.state[0, 5] == steps - 150
    two = torch.full((1, 100, 64), 2.0, device=dev)      # gates above 1 grow as they should
    assert torch.equal(det.det_gated_scan(two, torch.ones_like(two)).h[0, 99], torch.full((64,), 2.0 ** 100, device=dev))


def test_empty_sizes(dev):
    for shape in ((0, 5, 8), (3, 5, 0)):
        e = torch.empty(shape, device=dev)
        got = det.det_gated_scan(e, e)
        assert got.h.shape == shape and got.state.shape == (shape[0], shape[2])
        assert det.det_gated_scan_backward(e, e, e, e)[0].shape == shape
    with pytest.raises(det.DetError):
        det.det_gated_scan(torch.empty(2, 0, 8, device=dev), torch.empty(2, 0, 8, device=dev))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("ragged", [False, True])
def test_gradient_against_differences(dev, sigmoid, ragged):
    gate, x, state = inputs(3, 140, 9, torch.float32, dev, 4, sigmoid)
    lens = torch.tensor([140, 0, 77], dtype=torch.int32, device=dev) if ragged else None
    leaves = [v.requires_grad_(True) for v in (gate, x, state)]
    h, end = det.gated_scan(*leaves, sigmoid, lens)
    ch, ce = randn(h.shape, torch.float32, dev, 5), randn(end.shape, torch.float32, dev, 6)
    ((h * ch).sum() + (end * ce).sum()).backward()

    def value(g, u, s):
        hh, ee, _, _ = ref.scan(g, u, s, sigmoid, lens)
        return float((hh * ch.double()).sum() + (ee * ce.double()).sum())

    args = [v.detach().double() for v in leaves]
    for n, v in enumerate(leaves):
        step = randn(v.shape, torch.float32, dev, 30 + n).double()
        lo, hi = list(args), list(args)
        e = 1e-5
        lo[n], hi[n] = args[n] - e * step, args[n] + e * step
        slope = (value(*hi) - value(*lo)) / (2 * e)
        got = float((v.grad.double() * step).sum())
        size = float((v.grad.double() * step).abs().sum())
        assert abs(got - slope) <= 1e-5 * size + 1e-6, (n, got, slope)


def test_autograd_paths(dev):
    gate, x, state = inputs(2, 30, 20, torch.bfloat16, dev, 8, True)
    r = det.det_gated_scan(gate, x, state, True)
    ds = randn((2, 20), torch.float32, dev, 9)
    want = det.det_gated_scan_backward(torch.zeros_like(x), gate, x, r.h, state, ds, True)
    leaves = [v.clone().requires_grad_(True) for v in (gate, x, state)]
    det.gated_scan(*leaves, True)[1].backward(ds)      # the state alone
    for v, g in zip(leaves, want):
        assert same_bits(v.grad, g)
    a, b = gate.clone().requires_grad_(True), x.clone().requires_grad_(True)
    det.gated_scan(a, b, sigmoid=True)[0].sum().backward()      # h alone, a broadcast gradient
    r = det.det_gated_scan(gate, x, None, True)
    want = det.det_gated_scan_backward(torch.ones_like(x), gate, x, r.h, None, None, True)
    assert same_bits(a.grad, want[0]) and same_bits(b.grad, want[1])


def since_reset(x, reset):
    """Sums of x from the last reset on, whole numbers."""
    total = x.cumsum(0)
    at = torch.where(reset, torch.arange(len(x), device=x.device), torch.zeros_like(x)).cummax(0).values
    return total - total[at] + x[at]


def test_more_chunks_than_a_grid_holds(dev):
    """Whole numbers and gates of 0 and 1, so that every sum is exact; more than 2 * 65535 chunks."""
    n = 65536 * 128 + 77
    gate = torch.ones(n, device=dev)
    gate[torch.randint(0, n, (200,), generator=torch.Generator().manual_seed(1)).to(dev)] = 0
    x = torch.randint(-1, 2, (n,), generator=torch.Generator().manual_seed(2)).to(dev)
    dh = torch.zeros(n, dtype=torch.int64, device=dev)
    dh[::1009] = 1 - x[::1009]
    h = since_reset(x, gate == 0)
    got = det.det_gated_scan(gate.view(1, n, 1), x.float().view(1, n, 1))
    assert torch.equal(got.h.view(-1), h.float()) and got.state.item() == h[-1].item()
    resets = torch.cat([torch.ones(1, device=dev), gate.flip(0)[:-1]]) == 0
    g = since_reset(dh.flip(0), resets).flip(0)
    before = torch.cat([h.new_zeros(1), h[:-1]])
    assert (g * before).abs().max() < 2 ** 24
    dgate, dx, first = det.det_gated_scan_backward(dh.float().view(1, n, 1), gate.view(1, n, 1),
                                                   x.float().view(1, n, 1), got.h)
    assert torch.equal(dx.view(-1), g.float()) and torch.equal(dgate.view(-1), (g * before).float())


def test_more_sequences_than_a_grid_holds(dev):
    batch, steps = (1 << 22) + 5, 9
    gate = torch.randint(0, 2, (batch, steps, 1), generator=torch.Generator().manual_seed(3)).to(dev)
    x = torch.randint(-3, 4, (batch, steps, 1), generator=torch.Generator().manual_seed(4)).to(dev)
    lens = torch.arange(batch, dtype=torch.int32, device=dev) % 10
    state = x[:, 0] * 2
    h, now = torch.empty_like(x), state
    for i in range(steps):
        live = (i < lens)[:, None]
        now = torch.where(live, gate[:, i] * now + x[:, i], now)
        h[:, i] = torch.where(live, now, 0)
    got = det.det_gated_scan(gate.half(), x.half(), state.float(), lengths=lens)
    assert torch.equal(got.h, h.half()) and torch.equal(got.state, now.float())
    dgate, dx, first = det.det_gated_scan_backward(x.half(), gate.half(), x.half(), got.h, state.float(),
                                                   state.float(), lengths=lens)
    e, before = state, torch.cat([state[:, None], h[:, :-1]], 1)
    for i in reversed(range(steps)):
        live = (i < lens)[:, None]
        g = torch.where(live, x[:, i] + e, 0)
        assert torch.equal(dx[:, i], g.half()) and torch.equal(dgate[:, i], (g * before[:, i]).half())
        e = torch.where(live, gate[:, i] * g, e)
    assert torch.equal(first, e.float())
