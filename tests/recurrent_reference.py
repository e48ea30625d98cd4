"""Plain 64-bit statements of the embedding, layer norm, gated recurrence and linear cross entropy, and
running bounds of the recurrence's roundings.  They share no code with the library."""
import torch


def embedding(table, tokens, scale):
    known = (tokens >= 0) & (tokens < table.shape[0])
    rows = table.double()[torch.where(known, tokens, 0).long()] * scale
    return torch.where(known[..., None], rows, 0.0)


def embedding_backward(dout, tokens, vocab, scale):
    """(gradient, the sum of its terms' magnitudes)"""
    out = torch.zeros(2, vocab, dout.shape[-1], dtype=torch.float64, device=dout.device)
    d = dout.reshape(-1, dout.shape[-1]).double()
    for i, t in enumerate(tokens.reshape(-1).tolist()):
        if 0 <= t < vocab:
            out[0, t] += d[i]
            out[1, t] += d[i].abs()
    return out[0] * scale, out[1] * abs(scale)


def layer_norm(x, weight, bias, eps, residual=None):
    h = x.double() if residual is None else x.double() + residual.double()
    mean = h.mean(-1, keepdim=True)
    rstd = ((h - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    y = (h - mean) * rstd * weight.double()
    if bias is not None:
        y = y + bias.double()
    return h, mean[..., 0], rstd[..., 0], y


def layer_norm_backward(dy, h, weight, mean, rstd, dh=None):
    dy, w = dy.double(), weight.double()
    xhat = (h.double() - mean.double()[..., None]) * rstd.double()[..., None]
    g = dy * w
    dx = g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True)
    dx = dx * rstd.double()[..., None]
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy * xhat).flatten(0, -2).sum(0), dy.flatten(0, -2).sum(0)


def _terms(gate, x, sigmoid):
    """(a, b, relative error of each in units of 2^-24).  A sigmoid gate: e^-|gate| by the hardware is
    off by 2 (1 + |gate|), the addition by 1, the reciprocal by 2; b's product by 1."""
    g, u = gate.double(), x.double()
    if not sigmoid:
        return g, u, torch.zeros_like(g)
    a = torch.sigmoid(g)
    return a, torch.sigmoid(-g) * u, 6 + 2 * g.abs()


def scan(gate, x, state=None, sigmoid=False, lengths=None):
    """(h, state, bound of h, bound of state): the bounds in units of 2^-24 absolute."""
    a, b, r = _terms(gate, x, sigmoid)
    n, steps, d = a.shape
    h = torch.zeros(n, d, dtype=torch.float64, device=a.device) if state is None else state.double()
    m, e = h.abs(), torch.zeros_like(h)
    hs, es = torch.zeros_like(a), torch.zeros_like(a)
    for t in range(steps):
        live = torch.ones(n, 1, dtype=torch.bool, device=a.device)
        if lengths is not None:
            live = (t < lengths)[:, None]
        # a term that passes this step is multiplied once in its own chain and once in a product
        e1 = a[:, t].abs() * e + a[:, t].abs() * m * (r[:, t] + 2) + b[:, t].abs() * (r[:, t] + 2)
        m1 = a[:, t].abs() * m + b[:, t].abs()
        h1 = a[:, t] * h + b[:, t]
        h, m, e = torch.where(live, h1, h), torch.where(live, m1, m), torch.where(live, e1, e)
        # the effects of up to 16 spans composed, and the chunk's applied
        hs[:, t] = torch.where(live, h, 0.0)
        es[:, t] = torch.where(live, e + 40 * m, 0.0)
    return hs, h, es, e + 40 * m


def scan_backward(dh, gate, x, h, state=None, dstate=None, sigmoid=False, lengths=None):
    """(dgate, dx, first state's gradient), then their bounds in units of 2^-24 absolute."""
    a, _, r = _terms(gate, x, sigmoid)
    n, steps, d = a.shape
    grad = torch.zeros(n, d, dtype=torch.float64, device=a.device) if dstate is None else dstate.double()
    m, e = grad.abs(), torch.zeros_like(grad)
    first = torch.zeros_like(grad) if state is None else state.double()
    dg, dx, eg, ex = (torch.zeros_like(a) for _ in range(4))
    for t in range(steps - 1, -1, -1):
        live = torch.ones(n, 1, dtype=torch.bool, device=a.device)
        if lengths is not None:
            live = (t < lengths)[:, None]
        total, mt = grad + dh[:, t].double(), m + dh[:, t].double().abs()
        et = e + 40 * mt + mt
        before = h[:, t - 1].double() if t else first
        if sigmoid:
            keep, take = a[:, t], torch.sigmoid(-gate[:, t].double())
            i, g = take * total, keep * take * (before - x[:, t].double()) * total
            size = keep * take * (before.abs() + x[:, t].double().abs())
            ei, eg1 = take * (et + mt * (r[:, t] + 2)), size * (et + mt * (2 * r[:, t] + 5))
        else:
            i, g = total, before * total
            ei, eg1 = et, before.abs() * (et + mt)
        dx[:, t], dg[:, t] = torch.where(live, i, 0.0), torch.where(live, g, 0.0)
        ex[:, t], eg[:, t] = torch.where(live, ei, 0.0), torch.where(live, eg1, 0.0)
        e1 = a[:, t].abs() * (e + mt * (r[:, t] + 3))
        m1 = a[:, t].abs() * mt
        grad = torch.where(live, a[:, t] * total, grad)
        m, e = torch.where(live, m1, m), torch.where(live, e1, e)
    return dg, dx, grad, eg, ex, e + 40 * m


def xent(x, weight, targets, scale):
    """(loss, lse, logits, sums of the products' magnitudes)"""
    x, w = x.double(), weight.double()
    z, size = (x @ w.t()) * scale, (x.abs() @ w.abs().t()) * scale
    lse = torch.logsumexp(z, -1)
    on = (targets >= 0) & (targets < w.shape[0])
    picked = z.gather(-1, torch.where(on, targets, 0)[..., None])[..., 0]
    return torch.where(on, lse - picked, 0.0), lse, z, size


def xent_backward(x, weight, targets, lse, dloss, scale):
    """(dx, dweight, D, the rows' factors)"""
    z = xent(x, weight, targets, scale)[2]
    on = (targets >= 0) & (targets < weight.shape[0])
    d = torch.exp(z - lse.double()[:, None])
    d.scatter_add_(1, torch.where(on, targets, 0)[:, None], torch.full_like(d[:, :1], -1.0))
    d = torch.where(on[:, None], d, 0.0)
    f = torch.where(on, dloss.double() * scale, 0.0)[:, None]
    return (d * f) @ weight.double(), (d * f).t() @ x.double(), d, f
