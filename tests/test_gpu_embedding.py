"""det_embedding and the table's gradient on the GPU against 64-bit statements, at the token counts
where the sort changes (1024 tokens a chunk, 65536 in chunks), tokens met once, 64 and 65 times, all
the same, and outside the vocabulary.

Tolerances: a block of at most 64 rows is a chain of 63 additions, blocks join in 64 bits, one
rounding to f32, one by the scale and the type's half step."""
import pytest
import torch

import recurrent_reference as ref
from lm_reference import IDS, TYPES, U32, floor_of, half, randn, same_bits
from scan_fixed_order_amd import det

pytestmark = pytest.mark.gpu


def ids_of(n, vocab, dev, seed, kind="zipf", dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "same":
        t = torch.full((n,), vocab - 1)
    elif kind == "zipf":
        t = (torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * torch.log(torch.tensor(vocab + 0.0)))
             .long() - 1).clamp_(0, vocab - 1)
    else:
        t = torch.randint(0, vocab, (n,), generator=g)
    out = torch.randint(0, 9, (n,), generator=g)
    t = torch.where(out == 0, torch.tensor(-1), torch.where(out == 1, torch.tensor(vocab), t))
    return t.to(dtype).to(dev)


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("n,vocab,d", [(1, 1, 1), (1, 7, 3), (5, 10, 8), (64, 100, 129), (3, 9, 4097),
                                       (300, 50, 64), (9000, 33, 40), (17000, 5, 512), (2, 3, 20000)])
@pytest.mark.parametrize("scale", [1.0, 0.3])
def test_rows(dev, n, vocab, d, t, scale):
    table, ids = randn((vocab, d), t, dev, d), ids_of(n, vocab, dev, n, "even")
    got = det.det_embedding(table, ids, scale)
    want = ref.embedding(table, ids, scale)
    if scale == 1.0:
        assert same_bits(got, want.to(t))
    else:      # the scale is a float, the product one
        assert ((got.double() - want).abs() <= want.abs() * (half(t) + 2 * U32) * 1.001 + floor_of(t)).all()
    assert same_bits(got, det.det_embedding(table, ids.int(), scale))


def test_rows_views_shapes_and_special_values(dev):
    t = torch.bfloat16
    wide = randn((20, 71), t, dev, 1)
    wide[4, 9], wide[5, 10] = float("nan"), float("inf")
    table, ids = wide[:, 3:68], torch.tensor([[4, 5, -1], [19, 20, 0]], device=dev)
    got = det.det_embedding(table, ids)
    assert got.shape == (2, 3, 65) and got[0, 0, 6].isnan() and got[0, 1, 7].isinf()
    assert (got[0, 2] == 0).all() and (got[1, 1] == 0).all() and same_bits(got[1, 0], table[19].contiguous())
    big = torch.tensor([1 << 40, -(1 << 40), (1 << 32) + 4, 3], device=dev)      # no wrapping to 4
    assert (det.det_embedding(table, big)[:3] == 0).all()
    assert det.det_embedding(table[:0], ids).eq(0).all()
    assert det.det_embedding(table, ids[:0]).shape == (0, 3, 65)
    assert det.det_embedding(table[:, :0], ids).shape == (2, 3, 0)
    assert det.det_embedding(table, ids[0, 0]).shape == (65,)


GRAD = [(1, 1, 1, "even"), (5, 3, 7, "even"), (64, 40, 129, "same"), (65, 40, 129, "same"),
        (129, 4, 64, "same"), (700, 90, 65, "zipf"), (1024, 300, 24, "zipf"), (1025, 300, 24, "even"),
        (5000, 2000, 33, "zipf"), (9217, 64, 520, "zipf"), (20000, 1, 8, "same"), (65536, 700, 8, "zipf"),
        (65537, 700, 8, "zipf"), (70000, 70000, 5, "zipf"), (3, 9, 4097, "same"), (90, 3, 1030, "zipf")]


@pytest.mark.parametrize("t", TYPES, ids=IDS)
@pytest.mark.parametrize("n,vocab,d,kind", GRAD)
def test_table_gradient(dev, n, vocab, d, kind, t):
    ids, dout = ids_of(n, vocab, dev, n + d, kind), randn((n, d), t, dev, d)
    scale = 1.0 if n % 2 else 0.25
    got = det.det_embedding_backward(dout, ids, vocab, scale)
    cpu, size = ref.embedding_backward(dout.cpu(), ids.cpu(), vocab, scale)
    bound = 67 * U32 * size + half(t) * cpu.abs() * 1.001 + floor_of(t)
    assert ((got.double().cpu() - cpu).abs() <= bound).all()
    # the other token type, a strided dout, and again
    wide = torch.full((n, d + 3), float("nan"), device=dev).to(t)
    wide[:, 1:d + 1] = dout
    assert same_bits(got, det.det_embedding_backward(wide[:, 1:d + 1], ids.int(), vocab, scale))


def test_a_tokens_sum_depends_on_its_own_places_alone(dev):
    """Other tokens' places, their number (and with it the sort) and the vocabulary move no bit."""
    t, d = torch.float32, 72
    mine = randn((200, d), t, dev, 1)
    alone = det.det_embedding_backward(mine, torch.full((200,), 5, device=dev), 9)
    for n, vocab in ((300, 9), (5000, 400), (80000, 400)):
        ids = ids_of(n, vocab, dev, n, "even")
        ids[ids == 5] = 6
        at = torch.randperm(n, generator=torch.Generator().manual_seed(n))[:200].sort().values.to(dev)
        ids[at] = 5
        dout = randn((n, d), t, dev, n)
        dout[at] = mine
        got = det.det_embedding_backward(dout, ids, vocab)
        assert same_bits(got[5], alone[5])


def test_no_tokens_and_special_values(dev):
    t = torch.float16
    none = det.det_embedding_backward(torch.empty(0, 24, dtype=t, device=dev),
                                      torch.empty(0, dtype=torch.int64, device=dev), 70)
    assert none.shape == (70, 24) and (none == 0).all()
    ids = torch.tensor([-1, 70, 1 << 40, -7], device=dev)
    junk = torch.full((4, 24), float("nan"), device=dev).to(t)
    assert (det.det_embedding_backward(junk, ids, 70) == 0).all()      # of tokens that do not count
    ids = torch.tensor([1, 2, 1, 3], device=dev)
    dout = torch.ones(4, 24, dtype=t, device=dev)
    dout[0, 2], dout[3, 4] = float("nan"), float("inf")
    got = det.det_embedding_backward(dout, ids, 5)
    assert got[1, 2].isnan() and (got[1, 3:] == 2).all() and got[3, 4].isinf() and (got[2] == 1).all()
    assert det.det_embedding_backward(dout, ids, 0).shape == (0, 24)
    assert det.det_embedding_backward(dout[:, :0], ids, 5).shape == (5, 0)
    # sums past f16 stay sums until the one rounding
    many = torch.full((300, 8), 30000.0, device=dev).to(t)
    assert (det.det_embedding_backward(many, torch.zeros(300, dtype=torch.int64, device=dev), 2,
                                       scale=1 / 300)[0] == 30000).all()


def test_autograd(dev):
    t, vocab, d = torch.float32, 30, 20
    table = randn((vocab, d), t, dev, 1).requires_grad_(True)
    ids = ids_of(48, vocab, dev, 2, "zipf").view(6, 8)
    c = randn((6, 8, d), t, dev, 3)
    (det.embedding(table, ids, 0.5) * c).sum().backward()
    assert same_bits(table.grad, det.det_embedding_backward(c, ids, vocab, 0.5))
    table.grad = None
    det.embedding(table, ids).sum().backward()      # a broadcast gradient: the counts
    count = torch.bincount(ids[(ids >= 0) & (ids < vocab)], minlength=vocab)
    assert torch.equal(table.grad, count[:, None].expand(vocab, d).float())
