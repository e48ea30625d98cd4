"""Arguments of the language-model operators that would make a kernel read or write what is not
its own, refused before anything is enqueued; checked without a GPU."""
import pytest
import torch

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
