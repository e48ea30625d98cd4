"""The recurrent model's operators where a shortcut, a grid's bound or a sum's order could show: gates
that are not finite beside a state of zero."""
import pytest
import torch

from lm_reference import IDS, TYPES
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
