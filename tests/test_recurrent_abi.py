"""Refusals of the embedding, layer norm, gated recurrence and linear cross entropy, checked without
a GPU: through the C interface with addresses that are never dereferenced, and through the binding
with host tensors."""
import ctypes

import pytest
import torch

from scan_fixed_order_amd import det
from test_lm_abi import BF16, E4M3, F16, F32, F64, I32, INVALID, TOO_LARGE, UNSUPPORTED, WORKSPACE, at

I64 = 6
BIG = 1 << 35
off = ctypes.c_void_p


def embed(table=at(0), st=128, tok=at(1), tt=I64, n=5, v=100, d=128, t=BF16, scale=1.0, out=at(2)):
    return det.lib().det_embedding(table, st, tok, tt, n, v, d, t, scale, out, None)


def embed_back(dout=at(0), st=128, tok=at(1), tt=I64, n=5, v=100, d=128, t=BF16, scale=1.0,
               dtable=at(2), ws=at(3), nb=BIG):
    return det.lib().det_embedding_backward(dout, st, tok, tt, n, v, d, t, scale, dtable, ws, nb, None)


def layer(x=at(0), xs=128, res=at(1), rs=128, w=at(2), b=at(3), rows=4, d=128, t=BF16, eps=1e-5,
          h=at(4), y=at(5), mean=at(6), rstd=at(7)):
    return det.lib().det_layer_norm(x, xs, res, rs, w, b, rows, d, t, eps, h, y, mean, rstd, None)


def layer_back(dy=at(0), dys=128, h=at(1), hs=128, w=at(2), mean=at(3), rstd=at(4), dh=at(5), dhs=128,
               rows=4, d=128, t=BF16, dx=at(6), dw=at(7), db=at(8), ws=at(9), nb=BIG):
    return det.lib().det_layer_norm_backward(dy, dys, h, hs, w, mean, rstd, dh, dhs, rows, d, t, dx, dw,
                                             db, ws, nb, None)


def scan(gate=at(0), x=at(1), s0=at(2), lens=at(3), flags=1, batch=2, steps=20, d=128, t=BF16, h=at(4),
         s=at(5), ws=at(6), nb=BIG):
    return det.lib().det_gated_scan(gate, x, s0, lens, flags, batch, steps, d, t, h, s, ws, nb, None)


def scan_back(dh=at(0), gate=at(1), x=at(2), h=at(3), s0=at(4), ds=at(5), lens=at(6), flags=1, batch=2,
              steps=20, d=128, t=BF16, dg=at(7), dx=at(8), ds0=at(9), ws=at(10), nb=BIG):
    return det.lib().det_gated_scan_backward(dh, gate, x, h, s0, ds, lens, flags, batch, steps, d, t, dg,
                                             dx, ds0, ws, nb, None)


def xent(x=at(0), xs=128, w=at(1), wst=128, tg=at(2), rows=4, v=100, d=128, t=BF16, scale=1.0,
         loss=at(3), lse=at(4), ws=at(5), nb=BIG):
    return det.lib().det_linear_cross_entropy(x, xs, w, wst, tg, rows, v, d, t, scale, loss, lse, ws, nb,
                                              None)


def xent_back(x=at(0), xs=128, w=at(1), wst=128, tg=at(2), lse=at(3), dl=at(4), rows=4, v=100, d=128,
              t=BF16, scale=1.0, dx=at(5), dw=at(6), ws=at(7), nb=BIG):
    return det.lib().det_linear_cross_entropy_backward(x, xs, w, wst, tg, lse, dl, rows, v, d, t, scale,
                                                       dx, dw, ws, nb, None)


EVERY = [embed, embed_back, layer, layer_back, scan, scan_back, xent, xent_back]


@pytest.mark.parametrize("call", EVERY)
@pytest.mark.parametrize("t", [F64, I32, I64, E4M3, 9])
def test_types(call, t):
    assert call(t=t) == UNSUPPORTED


def test_other_operations_refuse_the_token_type():
    lib = det.lib()
    assert lib.det_sum(at(0), 10, I64, at(1), at(2), BIG, None) == UNSUPPORTED
    assert lib.det_scan(at(0), at(1), 10, I64, 0, None, 0, at(2), BIG, None) == UNSUPPORTED


def refused(call, what, bads):
    for bad in bads:
        assert call(**bad) == what, (call.__name__, bad)


def test_embedding_refusals():
    refused(embed, INVALID, [
        dict(table=None), dict(tok=None), dict(out=None), dict(st=127), dict(st=-1), dict(n=-1),
        dict(v=-1), dict(d=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e300),
        dict(table=off(at(0).value + 1)), dict(tok=off(at(1).value + 4)), dict(out=off(at(2).value + 1)),
        dict(tt=I32, tok=off(at(1).value + 2)), dict(out=at(0)), dict(out=off(at(0).value + 25000)),
        dict(out=at(1)), dict(out=off(at(1).value + 32))])
    refused(embed, UNSUPPORTED, [dict(tt=F32), dict(tt=BF16), dict(tt=7)])
    refused(embed, TOO_LARGE, [dict(n=1 << 31), dict(v=1 << 31), dict(d=1 << 31, st=1 << 31),
                               dict(st=1 << 61)])
    assert embed(n=0) == 0 and embed(d=0) == 0
    refused(embed_back, INVALID, [
        dict(dout=None), dict(tok=None), dict(dtable=None), dict(st=127), dict(n=-1), dict(v=-1),
        dict(d=-1), dict(scale=float("nan")), dict(dout=off(at(0).value + 1)),
        dict(tok=off(at(1).value + 4)), dict(dtable=off(at(2).value + 1)), dict(dtable=at(0)),
        dict(dtable=at(1)), dict(dtable=off(at(0).value - 25598))])
    refused(embed_back, UNSUPPORTED, [dict(tt=F32), dict(tt=7)])
    refused(embed_back, TOO_LARGE, [dict(n=1 << 31), dict(v=(1 << 31) - 1), dict(st=1 << 61)])
    refused(embed_back, WORKSPACE, [dict(ws=None), dict(nb=100), dict(ws=off(at(3).value + 128))])
    assert embed_back(v=0) == 0 and embed_back(d=0) == 0
    size = det.lib().det_embedding_backward_workspace_size
    assert size(5, 100, 128, BF16) > 0
    for bad in ((-1, 100, 128, BF16), (5, -1, 128, BF16), (5, 100, -1, BF16), (5, 100, 128, F64),
                (1 << 31, 100, 128, BF16), (5, 1 << 31, 128, BF16)):
        assert size(*bad) == 0


def test_layer_norm_refusals():
    refused(layer, INVALID, [
        dict(x=None), dict(w=None), dict(y=None), dict(h=None), dict(res=None), dict(xs=127),
        dict(rs=0), dict(xs=-1), dict(rows=-1), dict(d=-1), dict(d=0), dict(eps=-1.0),
        dict(eps=float("nan")), dict(eps=float("inf")), dict(x=off(at(0).value + 1)),
        dict(res=off(at(1).value + 1)), dict(w=off(at(2).value + 1)), dict(b=off(at(3).value + 1)),
        dict(h=off(at(4).value + 1)), dict(y=off(at(5).value + 1)), dict(mean=off(at(6).value + 2)),
        dict(rstd=off(at(7).value + 1))])
    # what is written may not lie over what is read, nor over each other
    refused(layer, INVALID, [
        dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3)), dict(y=at(4)), dict(h=at(2)),
        dict(h=at(3)), dict(h=off(at(0).value + 64)), dict(h=at(0), xs=256), dict(mean=at(7)),
        *[{name: at(i)} for name in ("mean", "rstd") for i in range(6)]])
    refused(layer, TOO_LARGE, [dict(rows=1 << 31), dict(d=1 << 31, xs=1 << 31, rs=1 << 31),
                               dict(xs=1 << 61)])
    assert layer(rows=0) == 0
    refused(layer_back, INVALID, [
        dict(dy=None), dict(h=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(dx=None),
        dict(dw=None), dict(dys=127), dict(hs=0), dict(dhs=5), dict(rows=-1), dict(d=0),
        dict(dx=at(2)), dict(dx=at(3)), dict(dx=at(4)), dict(db=at(7)), dict(dx=at(0), dys=256),
        dict(dx=off(at(1).value + 2)), dict(dx=at(0), d=16385, dys=16385, hs=16385, dhs=16385),
        dict(db=off(at(8).value + 1)),
        *[{name: at(i)} for name in ("dw", "db") for i in range(7)]])
    refused(layer_back, TOO_LARGE, [dict(rows=1 << 31)])
    refused(layer_back, WORKSPACE, [dict(ws=None), dict(nb=100), dict(ws=off(at(9).value + 128))])
    size = det.lib().det_layer_norm_backward_workspace_size
    assert size(16384, 4096, BF16) >= 2 * 4096 * 4
    assert size(-1, 8, BF16) == 0 and size(8, -1, BF16) == 0 and size(8, 8, F64) == 0


def test_gated_scan_refusals():
    refused(scan, INVALID, [
        dict(gate=None), dict(x=None), dict(h=None), dict(s=None), dict(flags=2), dict(batch=-1),
        dict(steps=-1), dict(d=-1), dict(steps=0), dict(gate=off(at(0).value + 1)),
        dict(x=off(at(1).value + 1)), dict(s0=off(at(2).value + 2)), dict(lens=off(at(3).value + 2)),
        dict(h=off(at(4).value + 1)), dict(s=off(at(5).value + 2)),
        *[dict(h=at(i)) for i in (0, 1, 2, 3, 5)], *[dict(s=at(i)) for i in (0, 1, 2, 3, 4)],
        dict(s=off(at(2).value + 4), steps=1), dict(h=at(2), steps=1)])
    refused(scan, TOO_LARGE, [dict(steps=1 << 31), dict(batch=1 << 16, d=1 << 16), dict(d=1 << 31),
                              dict(batch=1 << 31, d=0)])
    refused(scan, WORKSPACE, [dict(ws=None), dict(nb=100), dict(ws=off(at(6).value + 128))])
    assert scan(batch=0) == 0 and scan(d=0) == 0
    refused(scan_back, INVALID, [
        dict(dh=None), dict(gate=None), dict(x=None), dict(h=None), dict(dg=None), dict(dx=None),
        dict(flags=4), dict(batch=-1), dict(steps=0), dict(dh=off(at(0).value + 1)),
        dict(ds=off(at(5).value + 1)), dict(ds0=off(at(9).value + 1)),
        *[{name: at(i)} for name in ("dg", "dx", "ds0") for i in range(7)], dict(dg=at(8)),
        dict(dg=at(9)), dict(ds0=at(8))])
    refused(scan_back, TOO_LARGE, [dict(steps=1 << 31), dict(batch=1 << 16, d=1 << 16)])
    refused(scan_back, WORKSPACE, [dict(ws=None), dict(nb=100), dict(ws=off(at(10).value + 128))])
    for size in (det.lib().det_gated_scan_workspace_size, det.lib().det_gated_scan_backward_workspace_size):
        assert size(1, 32768, 64, BF16) >= 2 * 64 * 4 * 255
        for bad in ((-1, 8, 8, BF16), (8, -1, 8, BF16), (8, 8, -1, BF16), (8, 8, 8, F64),
                    (1 << 16, 8, 1 << 16, BF16)):
            assert size(*bad) == 0


def test_linear_cross_entropy_refusals():
    for call in (xent, xent_back):
        refused(call, INVALID, [
            dict(x=None), dict(w=None), dict(tg=None), dict(xs=127), dict(wst=5), dict(wst=-1),
            dict(rows=-1), dict(v=-1), dict(d=-1), dict(v=0), dict(d=0), dict(scale=0.0),
            dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-300),
            dict(x=off(at(0).value + 1)), dict(w=off(at(1).value + 1)), dict(tg=off(at(2).value + 4))])
        refused(call, TOO_LARGE, [dict(rows=(1 << 20) + 1), dict(v=1 << 31), dict(xs=1 << 61),
                                  dict(wst=1 << 61), dict(d=(1 << 20) + 1, xs=1 << 21, wst=1 << 21)])
        refused(call, WORKSPACE, [dict(ws=None), dict(nb=100)])
    refused(xent, INVALID, [
        dict(loss=None), dict(lse=None), dict(loss=at(4)), dict(loss=off(at(4).value + 12)),
        dict(loss=off(at(3).value + 2)), *[{n: at(i)} for n in ("loss", "lse") for i in range(3)]])
    refused(xent_back, INVALID, [
        dict(lse=None), dict(dl=None), dict(dx=None), dict(dw=None), dict(dx=at(6)),
        dict(dx=off(at(5).value + 1)), dict(lse=off(at(3).value + 1)), dict(dl=off(at(4).value + 2)),
        *[{n: at(i)} for n in ("dx", "dw") for i in range(5)]])
    assert xent(rows=0) == 0
    assert xent_back(rows=0, dw=None) == INVALID
    for size in (det.lib().det_linear_cross_entropy_workspace_size,
                 det.lib().det_linear_cross_entropy_backward_workspace_size):
        assert size(4, 100, 128, BF16) > 0
        for bad in ((-1, 100, 8, BF16), (4, -1, 8, BF16), (4, 100, -1, BF16), (4, 100, 8, F64),
                    (1 << 21, 100, 8, BF16), (4, 100, 1 << 21, BF16)):
            assert size(*bad) == 0


def test_binding_refuses_before_the_library():
    x, w, ids = torch.ones(4, 64), torch.ones(64), torch.zeros(4, dtype=torch.int64)
    table, bf = torch.ones(10, 64), x.bfloat16()
    s = torch.ones(2, 6, 32)
    for call in (lambda: det.det_layer_norm(x, w), lambda: det.det_embedding(table, ids),
                 lambda: det.det_embedding_backward(x, ids, 10), lambda: det.det_gated_scan(s, s),
                 lambda: det.det_gated_scan_backward(s, s, s, s),
                 lambda: det.det_linear_cross_entropy(x, table, ids),
                 lambda: det.det_linear_cross_entropy_backward(x, table, ids, w[:4], w[:4]),
                 lambda: det.det_layer_norm_backward(x, x, w, w[:4], w[:4])):
        with pytest.raises(ValueError, match="device tensors"):      # host tensors: no CPU path
            call()
    for call in (lambda: det.det_layer_norm(x.double(), w.double()), lambda: det.det_layer_norm(bf, w),
                 lambda: det.det_layer_norm(x, w, bias=w.half()),
                 lambda: det.det_layer_norm(x, w, residual=bf),
                 lambda: det.det_embedding(table, ids.float()), lambda: det.det_embedding(table.long(), ids),
                 lambda: det.det_embedding_backward(x, ids.short(), 10),
                 lambda: det.det_gated_scan(s, s.half()),
                 lambda: det.det_gated_scan(s, s, state=torch.ones(2, 32).half()),
                 lambda: det.det_gated_scan(s, s, lengths=torch.ones(2, dtype=torch.int64)),
                 lambda: det.det_gated_scan_backward(s, s, s, s.half()),
                 lambda: det.det_linear_cross_entropy(x, table.half(), ids),
                 lambda: det.det_linear_cross_entropy(x, table, ids.int()),
                 lambda: det.det_linear_cross_entropy_backward(x, table, ids, w[:4].double(), w[:4])):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: det.det_layer_norm(x, w[:63]), lambda: det.det_layer_norm(x, w, bias=w[:5]),
                 lambda: det.det_layer_norm(x, w, residual=torch.ones(3, 64)),
                 lambda: det.det_layer_norm(x.t(), torch.ones(4)),
                 lambda: det.det_layer_norm_backward(x, x, w, w[:3], w[:4]),
                 lambda: det.det_embedding(table[0], ids), lambda: det.det_embedding(table, ids[::2]),
                 lambda: det.det_embedding_backward(x, ids[:3], 10),
                 lambda: det.det_embedding_backward(x, ids, -1),
                 lambda: det.det_gated_scan(x, x), lambda: det.det_gated_scan(s, s[:, :5]),
                 lambda: det.det_gated_scan(s.transpose(0, 1), s.transpose(0, 1)),
                 lambda: det.det_gated_scan(s, s, state=torch.ones(2, 31)),
                 lambda: det.det_gated_scan(s, s, state_out=torch.ones(3, 32)),
                 lambda: det.det_gated_scan(s, s, lengths=torch.ones(3, dtype=torch.int32)),
                 lambda: det.det_gated_scan_backward(s, s, s, s[:1]),
                 lambda: det.det_linear_cross_entropy(x, table[:, :63], ids),
                 lambda: det.det_linear_cross_entropy(x, table, ids[:3]),
                 lambda: det.det_linear_cross_entropy(x, table[0], ids),
                 lambda: det.det_linear_cross_entropy_backward(x, table, ids, w[:3], w[:4]),
                 lambda: det.det_linear_cross_entropy_backward(x, table, ids, w[:4], w[:3])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("call", [
    lambda ws: det.det_layer_norm_backward(torch.ones(4, 64), torch.ones(4, 64), torch.ones(64),
                                           torch.ones(4), torch.ones(4), ws=ws),
    lambda ws: det.det_embedding_backward(torch.ones(4, 64), torch.zeros(4, dtype=torch.int32), 9, ws=ws),
    lambda ws: det.det_gated_scan(torch.ones(2, 6, 32), torch.ones(2, 6, 32), ws=ws),
    lambda ws: det.det_gated_scan_backward(*[torch.ones(2, 6, 32)] * 4, ws=ws),
    lambda ws: det.det_linear_cross_entropy(torch.ones(4, 64), torch.ones(9, 64),
                                            torch.zeros(4, dtype=torch.int64), ws=ws),
    lambda ws: det.det_linear_cross_entropy_backward(torch.ones(4, 64), torch.ones(9, 64),
                                                     torch.zeros(4, dtype=torch.int64), torch.ones(4),
                                                     torch.ones(4), ws=ws)])
def test_workspaces_without_memory_of_their_own(call):
    for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 20),
               torch.empty(1 << 21, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call(ws)


def test_gated_scan_takes_rows_up_to_a_width():
    wide = 4194303      # DET_SCAN_MAX_CHANNELS
    for call, size in ((scan, det.lib().det_gated_scan_workspace_size),
                       (scan_back, det.lib().det_gated_scan_backward_workspace_size)):
        refused(call, TOO_LARGE, [dict(batch=1, d=wide + 1)])
        assert size(1, 8, wide, BF16) > 0 and size(1, 8, wide + 1, BF16) == 0
