"""Refusals of the language-model operators, checked without a GPU: through the C interface with
addresses that are never dereferenced, and through the binding with host tensors."""
import ctypes

import pytest
import torch

from scan_fixed_order_amd import det

INVALID, UNSUPPORTED, TOO_LARGE, WORKSPACE = 1, 2, 3, 4
F32, F64, I32, F16, BF16, E4M3 = 0, 1, 2, 3, 4, 5
BIG = 1 << 30


def at(i):
    return ctypes.c_void_p((i + 1) << 36)      # far apart from each other


def norm(x=at(0), xs=128, res=at(1), rs=128, w=at(2), rows=4, d=128, t=BF16, eps=1e-6, h=at(3),
         y=at(4), yt=BF16, group=0, scales=None, rstd=at(5)):
    return det.lib().det_rms_norm(x, xs, res, rs, w, rows, d, t, eps, h, y, yt, group, scales, rstd,
                                  None)


def norm_back(dy=at(0), dys=128, h=at(1), hs=128, w=at(2), rstd=at(3), dh=at(4), dhs=128, rows=4,
              d=128, t=BF16, dx=at(5), dw=at(6), ws=at(7), n=BIG):
    return det.lib().det_rms_norm_backward(dy, dys, h, hs, w, rstd, dh, dhs, rows, d, t, dx, dw, ws,
                                           n, None)


def bias(table=at(0), buckets=32, heads=4, dist=128, flags=0, batch=2, q=8, k=16, off=0, offs=at(1),
         lens=at(2), scores=at(3), sb=512, sh=128, sq=16, t=BF16, out=at(4)):
    return det.lib().det_relative_bias(table, buckets, heads, dist, flags, batch, q, k, off, offs,
                                       lens, scores, sb, sh, sq, t, out, None)


def bias_back(dout=at(0), sb=512, sh=128, sq=16, buckets=32, heads=4, dist=128, flags=0, batch=2,
              q=8, k=16, off=0, offs=at(1), lens=at(2), t=BF16, dtable=at(3), dscores=at(4),
              ws=at(5), n=BIG):
    return det.lib().det_relative_bias_backward(dout, sb, sh, sq, buckets, heads, dist, flags, batch,
                                                q, k, off, offs, lens, t, dtable, dscores, ws, n,
                                                None)


def logp(x=at(0), st=1000, tg=at(1), rows=4, v=1000, t=BF16, scale=1.0, lp=at(2), en=at(3),
         lse=at(4), top=5, tl=at(5), ti=at(6)):
    return det.lib().det_token_logprobs(x, st, tg, rows, v, t, scale, lp, en, lse, top, tl, ti, None)


def logp_back(x=at(0), st=1000, tg=at(1), lse=at(2), dlp=at(3), en=at(4), den=at(5), rows=4, v=1000,
              t=BF16, scale=1.0, dx=at(6), dst=1000):
    return det.lib().det_token_logprobs_backward(x, st, tg, lse, dlp, en, den, rows, v, t, scale, dx,
                                                 dst, None)


@pytest.mark.parametrize("call", [norm, norm_back, bias, bias_back, logp, logp_back])
@pytest.mark.parametrize("t", [F64, I32, E4M3, 9])
def test_types(call, t):
    assert call(t=t) == UNSUPPORTED


def test_sums_and_scatters_refuse_the_storage_types():
    lib = det.lib()
    for t in (F16, BF16, E4M3):
        assert lib.det_sum(at(0), 10, t, at(1), at(2), BIG, None) == UNSUPPORTED
        assert lib.det_scan(at(0), at(1), 10, t, 0, None, 0, at(2), BIG, None) == UNSUPPORTED
        assert lib.det_scatter_add(at(0), at(1), 10, 1, t, at(2), 4, None, None, at(3), BIG,
                                   None) == UNSUPPORTED


def test_norm_refusals():
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(h=None), dict(res=None),
                dict(xs=127), dict(rs=0), dict(xs=-1), dict(rows=-1), dict(d=-1), dict(d=0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(group=32),
                dict(scales=at(6)), dict(yt=E4M3), dict(yt=E4M3, scales=at(6), group=16),
                dict(yt=E4M3, scales=at(6), group=256), dict(yt=E4M3, scales=at(6), group=-1)):
        assert norm(**bad) == INVALID, bad
    assert norm(yt=F32) == UNSUPPORTED
    assert norm(rows=1 << 31) == TOO_LARGE and norm(d=1 << 31, xs=1 << 31, rs=1 << 31) == TOO_LARGE
    assert norm(xs=1 << 61) == TOO_LARGE
    off = ctypes.c_void_p
    for bad in (dict(x=off(at(0).value + 1)), dict(res=off(at(1).value + 1)),
                dict(w=off(at(2).value + 1)), dict(h=off(at(3).value + 1)),
                dict(y=off(at(4).value + 1)), dict(rstd=off(at(5).value + 2)),
                dict(yt=E4M3, scales=off(at(6).value + 2))):
        assert norm(**bad) == INVALID, bad
    # what is written may not lie over what is read, nor over each other
    for bad in (dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3)), dict(h=at(2)),
                dict(h=off(at(0).value + 64)), dict(h=at(0), xs=256), dict(rstd=at(0)),
                dict(rstd=at(3)), dict(rstd=at(4)), dict(yt=E4M3, scales=at(4)),
                dict(yt=E4M3, scales=at(5)), dict(yt=E4M3, scales=at(1))):
        assert norm(**bad) == INVALID, bad
    assert norm(rows=0) == 0


def test_norm_backward_refusals():
    for bad in (dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None), dict(dx=None),
                dict(dw=None), dict(dys=127), dict(hs=0), dict(dhs=5), dict(rows=-1), dict(d=0),
                dict(dx=at(2)), dict(dw=at(0)), dict(dw=at(5)), dict(dw=at(2)), dict(dx=at(3)),
                dict(dx=ctypes.c_void_p(at(1).value + 2)), dict(dx=at(0), dys=256),
                dict(dx=at(0), d=16385, dys=16385, hs=16385, dhs=16385)):
        assert norm_back(**bad) == INVALID, bad
    assert norm_back(rows=1 << 31) == TOO_LARGE
    for bad in (dict(ws=None), dict(n=100), dict(ws=ctypes.c_void_p(at(7).value + 128))):
        assert norm_back(**bad) == WORKSPACE, bad
    size = det.lib().det_rms_norm_backward_workspace_size
    assert size(16384, 4096, BF16) >= 4096 * 4
    assert size(-1, 8, BF16) == 0 and size(8, -1, BF16) == 0 and size(8, 8, F64) == 0


def test_bias_refusals():
    for call in (bias, bias_back):
        for bad in (dict(flags=4), dict(batch=-1), dict(q=-1), dict(k=-1), dict(heads=0),
                    dict(buckets=0), dict(buckets=1), dict(buckets=2, flags=1),
                    dict(buckets=3, flags=1), dict(dist=16), dict(dist=0), dict(dist=-5),
                    dict(dist=8, flags=1), dict(off=1 << 41), dict(off=-(1 << 41)),
                    dict(offs=ctypes.c_void_p(at(1).value + 2)),
                    dict(lens=ctypes.c_void_p(at(2).value + 1)), dict(sb=-1), dict(sh=-1),
                    dict(sq=-1)):
            assert call(**bad) == INVALID, (call, bad)
        for bad in (dict(buckets=257, flags=1), dict(buckets=129), dict(heads=65536),
                    dict(batch=1 << 31), dict(q=1 << 31), dict(k=1 << 31), dict(dist=1 << 31),
                    dict(sb=1 << 61), dict(q=1 << 30, k=1 << 30, heads=64)):
            assert call(**bad) == TOO_LARGE, (call, bad)
    for bad in (dict(table=None), dict(out=None), dict(table=ctypes.c_void_p(at(0).value + 1)),
                dict(out=ctypes.c_void_p(at(4).value + 1)), dict(out=at(0)), dict(out=at(1)),
                dict(out=at(2)), dict(out=ctypes.c_void_p(at(3).value + 2)),
                dict(out=at(3), sb=1024), dict(scores=ctypes.c_void_p(at(3).value + 1))):
        assert bias(**bad) == INVALID, bad
    for empty in (dict(batch=0), dict(q=0), dict(k=0)):
        assert bias(**empty) == 0
    for bad in (dict(dout=None), dict(dtable=None), dict(dtable=at(0)), dict(dscores=at(3)),
                dict(dscores=at(0), sq=32), dict(dout=ctypes.c_void_p(at(0).value + 1))):
        assert bias_back(**bad) == INVALID, bad
    for bad in (dict(ws=None), dict(n=8), dict(ws=ctypes.c_void_p(at(5).value + 64))):
        assert bias_back(**bad) == WORKSPACE, bad
    size = det.lib().det_relative_bias_backward_workspace_size
    assert size(2, 4, 8, 16, 32, BF16) > 0 and size(2, 4, 8, 16, 257, BF16) == 0
    assert size(2, 0, 8, 16, 32, BF16) == 0 and size(-1, 4, 8, 16, 32, BF16) == 0


def test_logprob_refusals():
    for bad in (dict(x=None), dict(tg=None), dict(lp=None), dict(en=None), dict(lse=None),
                dict(tl=None), dict(ti=None), dict(top=0), dict(top=-1), dict(top=65),
                dict(top=6, v=5, st=5), dict(v=0, top=0, tl=None, ti=None), dict(rows=-1),
                dict(v=-1), dict(st=999), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e300),
                dict(scale=1e-300), dict(lp=at(0)), dict(tl=at(0)), dict(ti=at(0)),
                dict(x=ctypes.c_void_p(at(0).value + 1)), dict(tg=ctypes.c_void_p(at(1).value + 4)),
                dict(ti=ctypes.c_void_p(at(6).value + 4)), dict(lse=ctypes.c_void_p(at(4).value + 2))):
        assert logp(**bad) == INVALID, bad
    assert logp(v=(1 << 20) + 1, st=1 << 21) == TOO_LARGE
    assert logp(rows=1 << 31) == TOO_LARGE and logp(st=1 << 61) == TOO_LARGE
    assert logp(rows=0) == 0 and logp_back(rows=0) == 0
    for bad in (dict(x=None), dict(tg=None), dict(lse=None), dict(dlp=None), dict(en=None),
                dict(dx=None), dict(st=5), dict(dst=5), dict(v=0), dict(rows=-1), dict(scale=0.0),
                dict(dx=at(1)), dict(dx=at(2)), dict(dx=at(0), dst=2000),
                dict(dx=ctypes.c_void_p(at(0).value + 2)), dict(dx=ctypes.c_void_p(at(6).value + 1))):
        assert logp_back(**bad) == INVALID, bad
    assert logp_back(rows=1 << 31) == TOO_LARGE


def test_binding_refuses_before_the_library():
    x, w = torch.ones(4, 64), torch.ones(64)
    bf, d64 = x.bfloat16(), x.double()
    with pytest.raises(ValueError):
        det.det_rms_norm(x, w)                                   # host tensors: no CPU path
    with pytest.raises(TypeError):
        det.det_rms_norm(d64, w.double())
    with pytest.raises(TypeError):
        det.det_rms_norm(bf, w)                                  # weight of another type
    with pytest.raises(TypeError):
        det.det_rms_norm(x, w, residual=bf)
    with pytest.raises(TypeError):
        det.det_rms_norm(x, w, quant=torch.float8_e5m2)
    for bad in (dict(weight=torch.ones(63)), dict(residual=torch.ones(4, 63)), dict(group=32),
                dict(quant=torch.float8_e4m3fn, group=48)):
        with pytest.raises(ValueError):
            det.det_rms_norm(x, **{"weight": w, **bad})
    with pytest.raises(ValueError):
        det.det_rms_norm(x.t(), torch.ones(4))                   # rows not contiguous
    with pytest.raises(ValueError):
        det.det_rms_norm(x[:1].expand(3, 64), w)                 # rows over each other
    with pytest.raises(ValueError):
        det.det_rms_norm_backward(x, x, w, torch.ones(3))
    with pytest.raises(TypeError):
        det.det_rms_norm_backward(bf, x, w, torch.ones(4))
    table = torch.ones(32, 4)
    with pytest.raises(ValueError):
        det.det_relative_bias(table[0], 8, 8)
    with pytest.raises(ValueError):
        det.det_relative_bias(table, 8, 8, scores=torch.ones(1, 3, 8, 8))
    with pytest.raises(TypeError):
        det.det_relative_bias(table, 8, 8, lengths=torch.ones(2))
    with pytest.raises(ValueError):
        det.det_relative_bias(table, 8, 8, lengths=torch.ones(2, dtype=torch.int32),
                              q_offset=torch.ones(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        det.det_relative_bias(table, 8, 8, out=torch.ones(2, 4, 8, 8))
    with pytest.raises(ValueError):
        det.det_relative_bias_backward(torch.ones(4, 8, 8), 32)
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        det.det_token_logprobs(x, ids.int())
    with pytest.raises(ValueError):
        det.det_token_logprobs(x, ids[:3])
    with pytest.raises(ValueError):
        det.det_token_logprobs_backward(x, ids, torch.ones(4), torch.ones(4), dentropy=torch.ones(4))
    with pytest.raises(TypeError):
        det.det_token_logprobs_backward(x, ids, torch.ones(4), torch.ones(4).double())


def test_row_strides():
    f = det._row_stride
    x = torch.empty(4, 6, 32)
    assert f(x, "x") == 32 and f(x[..., :20], "x") == 32 and f(x[:, :1, :20], "x") == 192
    assert f(x[0, 0], "x") == 32 and f(x[:1, :1, :5], "x") == 5
    for bad in (x[:, ::2].transpose(0, 1), x[..., ::2], x[:, :3]):
        with pytest.raises(ValueError):
            f(bad, "x")
