"""Edges of the language-model operators on the GPU: rows of no elements, values at the ends of
their types, sizes at the ends of a launch."""

import pytest
import torch

from lm_reference import IDS, TYPES
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
