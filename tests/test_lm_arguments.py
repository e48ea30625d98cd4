"""Arguments of the language-model operators that would make a kernel read or write what is not
its own, refused before anything is enqueued; checked without a GPU."""
import ctypes

import pytest
import torch

from test_lm_abi import E4M3, INVALID, at, bias_back, logp, norm, norm_back
from scan_fixed_order_amd import det


@pytest.mark.parametrize("call", [
    lambda ws: det.det_rms_norm_backward(torch.ones(4, 64), torch.ones(4, 64), torch.ones(64),
                                         torch.ones(4), ws=ws),
    lambda ws: det.det_relative_bias_backward(torch.ones(2, 3, 8, 8), 32, ws=ws)])
def test_workspaces_without_memory_of_their_own(call):
    # 2^20 bytes by its shape, one by its storage; and every second byte of a buffer
    for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 20),
               torch.empty(1 << 21, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call(ws)


def test_outputs_over_what_other_workgroups_read_or_write():
    """Through the C interface, with addresses that are never dereferenced."""
    off = ctypes.c_void_p
    for bad in (dict(rstd=at(2)), dict(rstd=off(at(2).value + 252)),
                dict(yt=E4M3, scales=at(2)), dict(yt=E4M3, scales=off(at(2).value + 8))):
        assert norm(**bad) == INVALID, bad
    for bad in (dict(dw=at(3)), dict(dw=off(at(3).value - 254))):
        assert norm_back(**bad) == INVALID, bad
    for bad in (dict(dtable=at(1)), dict(dtable=at(2)), dict(dscores=at(1)), dict(dscores=at(2)),
                dict(dscores=off(at(2).value - 2046))):
        assert bias_back(**bad) == INVALID, bad
    for name, other in (("lp", 1), ("en", 1), ("lse", 1), ("tl", 1), ("ti", 1), ("lp", 3), ("lp", 4),
                        ("en", 4), ("lp", 5), ("en", 6), ("lse", 5), ("ti", 5), ("tl", 6), ("tl", 2)):
        assert logp(**{name: at(other)}) == INVALID, (name, other)
    # of 4 rows, 16 bytes each of floats: neighbours are fine, an overlap by one is not
    near = off(at(2).value + 12)
    assert logp(en=near) == INVALID and logp(lse=near) == INVALID and logp(tl=near) == INVALID
    assert logp(lp=off(at(1).value + 28)) == INVALID
