"""The workspace of the linear cross entropy as the header states it, without a GPU."""
import pytest

from scan_fixed_order_amd import det

SIZES = [(1, 1, 1), (3, 5, 8), (64, 32768, 2048), (65, 32768, 2048), (600, 30000, 1000), (4096, 65536, 4096),
         (16384, 131072, 1024), (16385, 131072, 1024), (65536, 65536, 4096), (1 << 20, 50000, 64),
         (1 << 20, 100, 7), (130, 1 << 20, 257), (2, 300, 1 << 20)]


@pytest.mark.parametrize("t,s", [(det.DET_F32, 4), (det.DET_F16, 2), (det.DET_BF16, 2)])
@pytest.mark.parametrize("rows,vocab,d", SIZES)
def test_backward(rows, vocab, d, t, s):
    piece = min(vocab, max(4096, min(65536, (1 << 26) // rows)))
    by = {"d": rows * piece * s * (2 if s == 2 else 1), "x": rows * d * s,
          "weight": piece * d * s if s == 2 and rows > 64 else 0, "sums": 4 * rows * d}
    got = det.det_linear_cross_entropy_backward_workspace_size(rows, vocab, d, t)
    # up to 256 entries less in a piece, whose number is a whole one of tiles
    least = by["d"] * (piece - 256) // piece if piece > 256 else 0
    assert got >= least + by["x"] + by["sums"]
    more = rows + 64 + 64, piece + 64 + 64, d + 4      # rounded up, and apart from powers of two
    most = (more[0] * more[1] * s * (2 if s == 2 else 1) + more[0] * d * s
            + (more[1] * d * s if by["weight"] else 0) + max(4 * rows * more[2], 1 << 26) + 8 * 256)
    assert got <= most, (got, most)


@pytest.mark.parametrize("rows,vocab,d", SIZES)
def test_forward(rows, vocab, d):
    for t in (det.DET_F32, det.DET_F16, det.DET_BF16):
        got = det.det_linear_cross_entropy_workspace_size(rows, vocab, d, t)
        assert 8 * rows * -(-vocab // 256) <= got <= 8 * rows * -(-vocab // 64) + 4 * rows + 512
