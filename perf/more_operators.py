"""Cases of the operators that a recurrent language model adds to those of `operators.py`: the
embedding, layer norm, the gated linear recurrence and the cross entropy behind an output
projection, each forward and backward.

With `own` false, `run` computes them from elementary torch operations in 32 bits and rounds once
at the end; with `own` true it calls this library's kernels.  `exact` states the definitions once
more in 64 bits."""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-5


def listed():
    return [
        # a decoding batch's tokens: latency
        {"name": "embed_token", "op": "embed", "n": 64, "vocab": 32768, "d": 4096, "type": "bf16",
         "scale": 1.0},
        # a batch of prompts, rows scaled by the root of the width
        {"name": "embed_prompt", "op": "embed", "n": 16384, "vocab": 131072, "d": 4096,
         "type": "bf16", "scale": 64.0},
        # a training step's gradient of the table: few tokens are met often, most never
        {"name": "embed_backward", "op": "embed_backward", "n": 32768, "vocab": 65536, "d": 2048,
         "type": "bf16", "scale": 1.0},
        # one token through a block's norm: latency
        {"name": "layer_token", "op": "layer", "rows": 1, "d": 4096, "type": "bf16",
         "residual": True, "bias": True},
        # a training step's norm: forward, and the gradients of stream, weight and bias
        {"name": "layer_train", "op": "layer_train", "rows": 16384, "d": 4096, "type": "bf16",
         "residual": True, "bias": True},
        # the same for an odd width in f32, without residual and bias
        {"name": "layer_train_odd", "op": "layer_train", "rows": 1003, "d": 5001, "type": "f32",
         "residual": False, "bias": False},
        # a decoding batch's recurrence: one step from the kept state
        {"name": "scan_token", "op": "scan", "batch": 64, "t": 1, "d": 4096, "type": "bf16",
         "sigmoid": True, "ragged": False, "state": True},
        # a few long prompts of different lengths, decay and input given as they are
        {"name": "scan_prompt_odd", "op": "scan", "batch": 3, "t": 10007, "d": 2500, "type": "f32",
         "sigmoid": False, "ragged": True, "state": False},
        # a training step's recurrence, forward and backward
        {"name": "scan_train", "op": "scan_train", "batch": 8, "t": 2048, "d": 4096,
         "type": "bf16", "sigmoid": True, "ragged": False, "state": False},
        # one token's loss: the whole projection is read
        {"name": "xent_token", "op": "xent", "rows": 1, "vocab": 32768, "d": 4096, "type": "bf16",
         "scale": 1.0},
        # a text scored under a temperature, odd width and vocabulary
        {"name": "xent_score_odd", "op": "xent", "rows": 517, "vocab": 50021, "d": 1003,
         "type": "f16", "scale": 1.25},
        # a training step's loss with the gradients of the stream and of the projection
        {"name": "xent_train", "op": "xent_train", "rows": 4096, "vocab": 65536, "d": 4096,
         "type": "bf16", "scale": 1.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    d = _log_int(rng, lo, hi)
    return min(hi, -(-d // 64) * 64) if rng.random() < 0.6 else d


def draw(rng):
    op = rng.choice(["embed", "embed_backward", "layer", "layer_train", "scan", "scan_train",
                     "xent", "xent_train"])
    c = {"op": op, "type": rng.choice(["f32", "f16", "bf16"])}
    if op.startswith("embed"):
        c["d"] = _width(rng, 64, 8192)
        c["vocab"] = _log_int(rng, 1000, min(262144, (1 << 27) // c["d"]))
        c["n"] = _log_int(rng, 1, min(32768, (1 << 26) // c["d"]))
        c["scale"] = rng.choice([1.0, 8.0, 0.3])
    elif op.startswith("layer"):
        c["d"] = _width(rng, 64, 16384)
        c["rows"] = _log_int(rng, 1, min(16384, (1 << 25) // c["d"]))
        c["residual"], c["bias"] = rng.random() < 0.5, rng.random() < 0.5
    elif op.startswith("scan"):
        c["d"] = _width(rng, 64, 8192)
        c["batch"] = _log_int(rng, 1, 64)
        c["t"] = 1 if op == "scan" and rng.random() < 0.2 else _log_int(
            rng, 1, max(1, min(32768, (1 << 25) // (c["d"] * c["batch"]))))
        c["sigmoid"], c["ragged"] = rng.random() < 0.5, rng.random() < 0.5
        c["state"] = rng.random() < 0.5
    else:
        c["d"] = _width(rng, 64, 4096)
        c["vocab"] = _log_int(rng, 1000, 131072)
        c["rows"] = _log_int(rng, 1, max(1, min(4096, (1 << 38) // (c["d"] * c["vocab"]))))
        c["scale"] = rng.choice([1.0, 0.8, 1.25])
    return c


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t, op = _TYPES[c["type"]], c["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev)

    def below(n, *shape):
        return torch.randint(0, n, shape, generator=g, device=dev)

    s = {"case": c}
    if op.startswith("embed"):
        n, v, d = c["n"], c["vocab"], c["d"]
        # the r-th most frequent token comes up about 1 / r of the time; ids in no order
        rank = torch.exp(uniform(n).double() * math.log(v)).long().clamp_(1, v) - 1
        ids = torch.randperm(v, generator=g, device=dev)[rank]
        s["tokens"] = torch.where(below(16, n) == 0, -1, ids)      # padding
        if op == "embed":
            s["table"] = normal(v, d).to(t)
        else:
            s["dout"] = (1e-2 * normal(n, d)).to(t)
    elif op.startswith("layer"):
        rows, d = c["rows"], c["d"]
        # a residual stream's channels differ in size and lie off zero, a few by far
        size = torch.exp(0.5 * normal(d)) * (1 + 9 * (below(100, d) == 0))
        off = 0.5 * normal(d)
        s["weight"] = (1 + 0.2 * normal(d)).to(t)
        s["bias"] = (0.1 * normal(d)).to(t) if c["bias"] else None
        s["x"] = ((normal(rows, d) + off) * size).to(t)
        s["residual"] = (normal(rows, d) * size).to(t) if c["residual"] else None
        if op != "layer":
            s["dy"] = (1e-2 * normal(rows, d)).to(t)
            s["dh"] = (1e-2 * normal(rows, d)).to(t) if c["residual"] else None
    elif op.startswith("scan"):
        shape = b, n, d = c["batch"], c["t"], c["d"]
        # channels forget at their own rates, from a few steps to hundreds
        gate = normal(*shape).add_(1 + 1.5 * normal(d))
        s["gate"] = gate.to(t) if c["sigmoid"] else gate.sigmoid_().to(t)
        s["x"] = normal(*shape).to(t)
        s["state"] = normal(b, d) if c["state"] else None
        s["lengths"] = (n - below(max(1, n // 2), b)).to(torch.int32) if c["ragged"] else None
        if op != "scan":
            s["dh"] = (1e-2 * normal(*shape)).to(t)
            s["dstate"] = 1e-2 * normal(b, d) if c["state"] else None
    else:
        rows, v, d = c["rows"], c["vocab"], c["d"]
        targets = below(v, rows)
        weight = normal(v, d).mul_(2.5 / math.sqrt(d))
        s["weight"] = weight.to(t)
        # what a trained model knows of the next token: its logit stands out
        hit = weight[targets]
        s["x"] = (normal(rows, d) + hit * (8.0 / hit.square().sum(1, keepdim=True))).to(t)
        # an eighth of the positions belongs to the prompt or the padding
        s["targets"] = torch.where(below(8, rows) == 0, -100, targets)
        if op != "xent":
            s["dloss"] = torch.full((rows,), 1.0 / rows, device=dev) * (0.5 + uniform(rows))
    return s


# ------------------------------------------------------------------ plain forms

def _embed(s):
    table, tokens = s["table"], s["tokens"]
    known = (tokens >= 0) & (tokens < table.shape[0])
    rows = table[torch.where(known, tokens, 0)].float() * s["case"]["scale"]
    return torch.where(known[:, None], rows, 0.0).to(table.dtype)


def _embed_backward(s):
    c, tokens = s["case"], s["tokens"]
    known = (tokens >= 0) & (tokens < c["vocab"])
    # one row more takes what belongs to no token
    total = torch.zeros(c["vocab"] + 1, c["d"], device=tokens.device)
    total.index_add_(0, torch.where(known, tokens, c["vocab"]), s["dout"].float())
    return total[:-1].mul_(c["scale"]).to(s["dout"].dtype)


def _layer(s):
    t, h = s["x"].dtype, s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    mean = h.mean(1, keepdim=True)
    rstd = torch.rsqrt((h - mean).square().mean(1, keepdim=True) + _EPS)
    y = (h - mean) * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return h.to(t), mean, rstd, y.to(t)


def _layer_outputs(s, h, y):
    return {"y": y, "h": h} if s["residual"] is not None else {"y": y}


def _layer_backward(s, h, mean, rstd):
    t = h.dtype
    xhat = (h.float() - mean) * rstd
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    out = {"dx": dx.to(t), "dweight": (dy * xhat).sum(0).to(t)}
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0).to(t)
    return out


def _doubling(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dimension 1: spans of 1, 2, 4, ... steps joined."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat([b[:, :step], torch.addcmul(b[:, step:], a[:, step:], b[:, :-step])], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _inside(s):
    """Which steps belong to their sequence: [batch, t, 1], or None for all."""
    if s["lengths"] is None:
        return None
    return (torch.arange(s["case"]["t"], device=s["x"].device) < s["lengths"][:, None])[:, :, None]


def _scan_terms(s):
    """(decay, input) of every step in 32 bits; steps past a length keep the state."""
    gate, x = s["gate"].float(), s["x"].float()
    a, b = (gate.sigmoid(), gate.neg().sigmoid() * x) if s["case"]["sigmoid"] else (gate, x)
    inside = _inside(s)
    if inside is not None:
        a, b = torch.where(inside, a, 1.0), torch.where(inside, b, 0.0)
    return a, b


def _scan(s):
    a, b = _scan_terms(s)
    if s["state"] is not None:
        b = torch.cat([torch.addcmul(b[:, :1], a[:, :1], s["state"][:, None]), b[:, 1:]], 1)
    h = _doubling(a, b)
    state, inside = h[:, -1].clone(), _inside(s)
    if inside is not None:
        h = torch.where(inside, h, 0.0)
    return h, state


def _scan_backward(s, h):
    c, t, inside = s["case"], s["x"].dtype, _inside(s)
    a, _ = _scan_terms(s)
    dh = s["dh"].float()
    if inside is not None:
        dh = torch.where(inside, dh, 0.0)
    if s["dstate"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dstate"][:, None]], 1)
    # G[t] = dh[t] + a[t+1] G[t+1], from the last step on
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1).flip(1)
    grad = _doubling(after, dh.flip(1)).flip(1)
    dstate = (a[:, 0] * grad[:, 0]) if s["state"] is not None else None
    if inside is not None:
        grad = torch.where(inside, grad, 0.0)
    first = torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    if c["sigmoid"]:
        gate, x = s["gate"].float(), s["x"].float()
        keep, take = gate.sigmoid(), gate.neg().sigmoid()
        dgate, dx = keep * take * (before - x) * grad, take * grad
    else:
        dgate, dx = before * grad, grad
    out = {"dgate": dgate.to(t), "dx": dx.to(t)}
    if dstate is not None:
        out["dstate"] = dstate
    return out


def _xent(s):
    z = s["x"].float() @ s["weight"].float().t()
    z *= s["case"]["scale"]
    m = z.amax(1, keepdim=True)
    z -= m
    log_total = z.exp().sum(1, keepdim=True).log_()
    scored = s["targets"] >= 0
    picked = z.gather(1, torch.where(scored, s["targets"], 0)[:, None])
    loss = torch.where(scored, (log_total - picked)[:, 0], 0.0)
    return z, log_total, {"loss": loss, "lse": (m + log_total)[:, 0]}


def _xent_backward(s, z, log_total):
    t, scale = s["x"].dtype, s["case"]["scale"]
    scored = s["targets"] >= 0
    dloss = torch.where(scored, s["dloss"], 0.0)
    p = z.sub_(log_total).exp_().mul_(dloss[:, None])
    rows = torch.arange(p.shape[0], device=p.device)
    p[rows, torch.where(scored, s["targets"], 0)] -= dloss
    p *= scale
    return {"dx": (p @ s["weight"].float()).to(t), "dweight": (p.t() @ s["x"].float()).to(t)}


def _plain(s):
    op = s["case"]["op"]
    if op == "embed":
        return {"out": _embed(s)}
    if op == "embed_backward":
        return {"dtable": _embed_backward(s)}
    if op.startswith("layer"):
        h, mean, rstd, y = _layer(s)
        out = _layer_outputs(s, h, y)
        return out if op == "layer" else {**out, **_layer_backward(s, h, mean, rstd)}
    if op.startswith("scan"):
        h, state = _scan(s)
        out = {"h": h.to(s["x"].dtype), "state": state}
        return out if op == "scan" else {**out, **_scan_backward(s, h)}
    z, log_total, out = _xent(s)
    return out if op == "xent" else {**out, **_xent_backward(s, z, log_total)}


# ------------------------------------------------------------------ the library's calls

def _own(s):
    from scan_fixed_order_amd import det

    c = s["case"]
    op = c["op"]
    if op == "embed":
        return {"out": det.det_embedding(s["table"], s["tokens"], scale=c["scale"])}
    if op == "embed_backward":
        return {"dtable": det.det_embedding_backward(s["dout"], s["tokens"], c["vocab"],
                                                     scale=c["scale"])}
    if op.startswith("layer"):
        r = det.det_layer_norm(s["x"], s["weight"], bias=s["bias"], eps=_EPS,
                               residual=s["residual"])
        out = _layer_outputs(s, r.h, r.y)
        if op != "layer":
            dx, dweight, dbias = det.det_layer_norm_backward(s["dy"], r.h, s["weight"], r.mean,
                                                             r.rstd, dh=s["dh"])
            out.update(dx=dx, dweight=dweight)
            if s["bias"] is not None:
                out["dbias"] = dbias
        return out
    if op.startswith("scan"):
        how = {"sigmoid": c["sigmoid"], "lengths": s["lengths"]}
        r = det.det_gated_scan(s["gate"], s["x"], state=s["state"], **how)
        out = {"h": r.h, "state": r.state}
        if op != "scan":
            dgate, dx, dstate = det.det_gated_scan_backward(
                s["dh"], s["gate"], s["x"], r.h, state=s["state"], dstate=s["dstate"], **how)
            out.update(dgate=dgate, dx=dx)
            if s["state"] is not None:
                out["dstate"] = dstate
        return out
    r = det.det_linear_cross_entropy(s["x"], s["weight"], s["targets"], scale=c["scale"])
    out = {"loss": r.loss, "lse": r.lse}
    if op != "xent":
        out["dx"], out["dweight"] = det.det_linear_cross_entropy_backward(
            s["x"], s["weight"], s["targets"], r.lse, s["dloss"], scale=c["scale"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, e, op = case, _BYTES[case["type"]], case["op"]
    if op.startswith("embed"):
        n = c["n"] * c["d"]
        if op == "embed":
            return {"bytes": 2 * n * e + 8 * c["n"], "flops": n}
        return {"bytes": (n + c["vocab"] * c["d"]) * e + 8 * c["n"], "flops": n}
    if op.startswith("layer"):
        n, d, rows = c["rows"] * c["d"], c["d"], c["rows"]
        parts = 2 if c["bias"] else 1
        moved, flops = n * e * (4 if c["residual"] else 2) + parts * d * e, 8 * n
        if op != "layer":
            # h is what the forward pass wrote, x itself without a residual
            moved += n * e * (4 if c["residual"] else 3) + 2 * parts * d * e + 8 * rows
            flops += 14 * n
        return {"bytes": moved, "flops": flops}
    if op.startswith("scan"):
        cells = c["batch"] * c["d"]
        left = 0.75 if c["ragged"] else 1.0      # lengths lie between a half and the whole
        n = cells * c["t"] * e
        moved = left * 2 * n + n + 4 * cells * (2 if c["state"] else 1)
        flops = left * cells * c["t"] * (10 if c["sigmoid"] else 2)
        if op != "scan":
            streams = 4 if c["sigmoid"] else 3      # gate, h, dh, and x where the gate mixes it in
            moved += left * streams * n + 2 * n + (12 * cells if c["state"] else 0)
            flops *= 2.5
        return {"bytes": moved, "flops": flops}
    rows, v, d = c["rows"], c["vocab"], c["d"]
    moved, flops = (rows + v) * d * e + 16 * rows, 2 * rows * v * d + 4 * rows * v
    if op != "xent":
        moved += 2 * (rows + v) * d * e + 16 * rows
        flops += 4 * rows * v * d + 4 * rows * v
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_embed(s):
    out = torch.zeros(s["tokens"].shape[0], s["case"]["d"], dtype=torch.float64,
                      device=s["tokens"].device)
    at = torch.nonzero(s["tokens"] >= 0)[:, 0]
    out[at] = s["table"].index_select(0, s["tokens"][at]).double() * s["case"]["scale"]
    return {"out": out}


def _exact_embed_backward(s):
    c, order = s["case"], torch.argsort(s["tokens"], stable=True)
    ids = s["tokens"][order]
    order, ids = order[ids >= 0], ids[ids >= 0]
    out = torch.zeros(c["vocab"], c["d"], dtype=torch.float64, device=ids.device)
    # the sums of runs of equal tokens: differences of running sums over the sorted rows
    used, counts = torch.unique_consecutive(ids, return_counts=True)
    ends = counts.cumsum(0)
    for i in range(0, c["d"], 512):
        run = s["dout"][:, i:i + 512][order].double().cumsum(0)
        at = run[ends - 1]
        out[used, i:i + 512] = torch.diff(at, dim=0, prepend=torch.zeros_like(at[:1]))
    return {"dtable": out * c["scale"]}


def _exact_layer(s):
    c, h = s["case"], s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    var, mean = torch.var_mean(h, 1, correction=0, keepdim=True)
    n = (h - mean) / torch.sqrt(var + _EPS)
    y = n * s["weight"].double()
    if s["bias"] is not None:
        y = y + s["bias"].double()
    out = {"y": y, "h": h} if s["residual"] is not None else {"y": y}
    if c["op"] == "layer":
        return out
    # the gradient sees h as it is kept
    h = h.to(s["x"].dtype).double()
    n = (h - mean) / torch.sqrt(var + _EPS)
    dy = s["dy"].double()
    dn = dy * s["weight"].double()
    d = h.shape[1]
    dx = (d * dn - dn.sum(1, keepdim=True) - n * (dn * n).sum(1, keepdim=True))
    dx = dx / (d * torch.sqrt(var + _EPS))
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    out.update(dx=dx, dweight=torch.einsum("rd,rd->d", dy, n))
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _exact_scan(s):
    c = s["case"]
    b, n, d = c["batch"], c["t"], c["d"]
    gate, x = s["gate"].transpose(0, 1), s["x"].transpose(0, 1)
    live = torch.ones(n, b, 1, dtype=torch.bool, device=x.device)
    if s["lengths"] is not None:
        live = (torch.arange(n, device=x.device)[:, None] < s["lengths"][None])[:, :, None]
    a = gate.double()
    u = x.double()
    if c["sigmoid"]:
        a = 1 / (1 + torch.exp(-a))
        u = (1 - a) * u
    h = torch.zeros(b, d, dtype=torch.float64, device=x.device)
    if s["state"] is not None:
        h = s["state"].double()
    start, hs = h, torch.empty(n, b, d, dtype=torch.float64, device=x.device)
    for i in range(n):
        h = torch.where(live[i], a[i] * h + u[i], h)
        hs[i] = h
    out = {"h": torch.where(live, hs, 0.0).transpose(0, 1), "state": h}
    if c["op"] == "scan":
        return out
    grad = torch.zeros_like(h) if s["dstate"] is None else s["dstate"].double()
    dgate, dx = torch.zeros_like(hs), torch.zeros_like(hs)
    dh = s["dh"].transpose(0, 1)
    for i in range(n - 1, -1, -1):
        total = grad + dh[i].double()
        before = hs[i - 1] if i else start
        if c["sigmoid"]:
            dg = a[i] * (1 - a[i]) * (before - x[i].double()) * total
            di = (1 - a[i]) * total
        else:
            dg, di = before * total, total
        dgate[i], dx[i] = torch.where(live[i], dg, 0.0), torch.where(live[i], di, 0.0)
        grad = torch.where(live[i], a[i] * total, grad)
    out.update(dgate=dgate.transpose(0, 1), dx=dx.transpose(0, 1))
    if s["state"] is not None:
        out["dstate"] = grad
    return out


def _exact_xent(s):
    c, w = s["case"], s["weight"].double()
    train = c["op"] != "xent"
    loss, lses, dx = [], [], []
    dw = torch.zeros_like(w) if train else None
    for i in range(0, c["rows"], 1024):
        r = slice(i, i + 1024)
        x, at = s["x"][r].double(), s["targets"][r]
        z = torch.mm(x, w.t()) * c["scale"]
        lse = torch.logsumexp(z, 1)
        on = at >= 0
        hit = torch.zeros_like(z).scatter_(1, at.clamp_min(0)[:, None], 1.0)
        loss.append(torch.where(on, lse - (z * hit).sum(1), 0.0))
        lses.append(lse)
        if train:
            d = torch.exp(z - lse[:, None]) - hit
            d *= (torch.where(on, s["dloss"][r].double(), 0.0) * c["scale"])[:, None]
            dx.append(torch.mm(d, w))
            dw += torch.mm(d.t(), x)
    out = {"loss": torch.cat(loss), "lse": torch.cat(lses)}
    if train:
        out.update(dx=torch.cat(dx), dweight=dw)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        return _exact_embed(s)
    if op == "embed_backward":
        return _exact_embed_backward(s)
    if op.startswith("layer"):
        return _exact_layer(s)
    if op.startswith("scan"):
        return _exact_scan(s)
    return _exact_xent(s)
