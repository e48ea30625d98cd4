"""The language-model operators' cases: root-mean-square norm, relative position bias, token log
probabilities, each forward and backward.

With `own` false, `run` computes them from elementary torch operations in 32 bits (64 where 32
lose what matters) and rounds once at the end; with `own` true it calls this library's kernels.
`exact` states the definitions once more in 64 bits."""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_E4M3_MAX = 448.0
_TINY = 2.0 ** -100     # a group's largest magnitude below this counts as this
_EPS = 1e-6


def listed():
    return [
        # one token of a decoding step through a block's norm: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "d": 4096, "type": "bf16",
         "residual": True, "bits8": False, "group": 0},
        # a prompt's tokens on their way into an 8-bit projection, a scale for every 128 channels
        {"name": "norm_prompt_8bit", "op": "norm", "rows": 8192, "d": 8192, "type": "bf16",
         "residual": True, "bits8": True, "group": 128},
        # odd width, no residual, one scale a row
        {"name": "norm_odd_8bit", "op": "norm", "rows": 1003, "d": 5001, "type": "f16",
         "residual": False, "bits8": True, "group": 0},
        # a training step's norm backward: gradients of the stream and of the weight
        {"name": "norm_backward", "op": "norm_backward", "rows": 16384, "d": 4096, "type": "bf16",
         "residual": True},
        # a decoding batch, every sequence at its own position
        {"name": "bias_token", "op": "bias", "batch": 32, "heads": 16, "q": 1, "k": 4097,
         "type": "bf16", "buckets": 32, "distance": 128, "two_sided": False, "causal": True,
         "ragged": True, "scores": False},
        # an encoder's bias, made once for all its layers
        {"name": "bias_encoder", "op": "bias", "batch": 1, "heads": 16, "q": 4096, "k": 4096,
         "type": "bf16", "buckets": 32, "distance": 128, "two_sided": True, "causal": False,
         "ragged": False, "scores": False},
        # the table's gradient in a training step over a batch of full sequences
        {"name": "bias_backward", "op": "bias_backward", "batch": 4, "heads": 16, "q": 2048,
         "k": 2048, "type": "bf16", "buckets": 32, "distance": 128, "two_sided": True,
         "causal": False, "ragged": False, "scores": False},
        # a decoder's training step on padded sequences of odd lengths: scores plus bias, gradient
        {"name": "bias_train_odd", "op": "bias_train", "batch": 3, "heads": 5, "q": 777,
         "k": 1003, "type": "f32", "buckets": 32, "distance": 256, "two_sided": False,
         "causal": True, "ragged": True, "scores": True},
        # a sampled token of a single sequence, with the alternatives shown beside it
        {"name": "logp_token", "op": "logp", "rows": 1, "vocab": 32768, "type": "bf16", "top": 8,
         "scale": 1.0},
        # a long prompt scored for evaluation
        {"name": "logp_score", "op": "logp", "rows": 2048, "vocab": 131072, "type": "bf16",
         "top": 5, "scale": 1.0},
        # the gradient that a training step sends into the output projection
        {"name": "logp_backward", "op": "logp_backward", "rows": 4096, "vocab": 65536,
         "type": "bf16", "scale": 1.0},
        # policy training at a temperature on an odd vocabulary: log probabilities, entropy, gradient
        {"name": "logp_train_odd", "op": "logp_train", "rows": 517, "vocab": 50021, "type": "f32",
         "top": 0, "scale": 1.25},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "bias", "bias_backward", "bias_train",
                     "logp", "logp", "logp_backward", "logp_train"])
    c = {"op": op, "type": rng.choice(["f32", "f16", "bf16"])}
    if op.startswith("norm"):
        c["d"] = _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            c["d"] = -(-c["d"] // 128) * 128
        c["rows"] = _log_int(rng, 1, min(16384, (1 << 25) // c["d"]))
        c["residual"] = rng.random() < 0.5
        if op == "norm":
            c["bits8"] = rng.random() < 0.5
            c["group"] = rng.choice([0, 32, 64, 128]) if c["bits8"] else 0
    elif op.startswith("bias"):
        c["batch"], c["heads"] = rng.randint(1, 8), rng.randint(1, 24)
        c["k"] = _log_int(rng, 16, 4096)
        c["q"] = 1 if op == "bias" and rng.random() < 0.3 else _log_int(
            rng, 1, max(1, min(c["k"], (1 << 25) // (c["batch"] * c["heads"] * c["k"]))))
        c["buckets"] = rng.choice([16, 32, 64])
        c["distance"] = rng.choice([64, 100, 128, 256, 500, 1024])
        c["two_sided"] = rng.random() < 0.5
        c["causal"] = rng.random() < 0.5
        c["ragged"] = rng.random() < 0.5
        c["scores"] = op == "bias_train" or rng.random() < 0.5
    else:
        c["vocab"] = _log_int(rng, 1000, 262144)
        c["rows"] = _log_int(rng, 1, min(4096, (1 << 26) // c["vocab"]))
        c["scale"] = rng.choice([1.0, 0.8, 1.25])
        if op != "logp_backward":
            c["top"] = rng.choice([0, 1, 5, 20])
    return c


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = _TYPES[c["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def below(n, *shape):
        return torch.randint(0, n, shape, generator=g, device=dev)

    s = {"case": c}
    if c["op"].startswith("norm"):
        rows, d = c["rows"], c["d"]
        # a residual stream's channels differ in size, a few by an order of magnitude
        size = torch.exp(0.5 * normal(d)) * (1 + 9 * (below(100, d) == 0))
        s["weight"] = (1 + 0.2 * normal(d)).to(t)
        if c["op"] == "norm":
            s["x"] = (normal(rows, d) * size).to(t)
            s["residual"] = (normal(rows, d) * size).to(t) if c["residual"] else None
        else:
            h = normal(rows, d) * size
            s["h"] = h.to(t)
            s["rstd"] = torch.rsqrt(h.square().mean(1) + _EPS)
            s["dy"] = (1e-2 * normal(rows, d)).to(t)
            s["dh"] = (1e-2 * normal(rows, d)).to(t) if c["residual"] else None
    elif c["op"].startswith("bias"):
        b, h, q, k = c["batch"], c["heads"], c["q"], c["k"]
        s["table"] = normal(c["buckets"], h).to(t)
        s["q_offset"], s["lengths"] = k - q, None      # the last q of k positions ask
        if c["ragged"]:
            n = k - below(max(1, k // 2), b)
            s["lengths"] = n.to(torch.int32)
            if c["op"] == "bias" and q == 1:
                s["q_offset"] = (n - 1).to(torch.int32)
        s["scores"] = (2 * normal(b, h, q, k)).to(t) if c["scores"] else None
        if c["op"] != "bias":
            s["dout"] = (1e-3 * normal(b, h, q, k)).to(t)
    else:
        rows, vocab = c["rows"], c["vocab"]
        targets = below(vocab, rows)
        logits = 2.5 * normal(rows, vocab)
        logits[torch.arange(rows, device=dev), targets] += 8.0
        s["logits"] = logits.to(t)
        # an eighth of the positions belongs to the prompt and is not scored
        s["targets"] = torch.where(below(8, rows) == 0, -100, targets)
        if c["op"] != "logp":
            s["dlogp"], s["dentropy"] = normal(rows) / rows, 1e-2 * normal(rows) / rows
        if c["op"] == "logp_backward":
            logits.copy_(s["logits"]).mul_(c["scale"])
            s["lse"] = torch.logsumexp(logits, 1)
            logits.sub_(s["lse"][:, None])
            s["entropy"] = -(logits.exp() * logits).sum(1)
    return s


# ------------------------------------------------------------------ plain forms

def _norm(s):
    c, t = s["case"], s["x"].dtype
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + _EPS) * s["weight"].float()
    out = {"h": h.to(t)} if s["residual"] is not None else {}
    if not c["bits8"]:
        return {**out, "y": y.to(t)}
    rows, d = y.shape
    group = c["group"] or d
    blocks = torch.nn.functional.pad(y, (0, -d % group)).view(rows, -1, group)
    largest = blocks.abs().amax(2).clamp_min(_TINY)
    q = (blocks * (_E4M3_MAX / largest)[:, :, None]).reshape(rows, -1)[:, :d]
    return {**out, "y": q.to(torch.float8_e4m3fn), "scales": largest / _E4M3_MAX}


def _norm_backward(s):
    t, d = s["h"].dtype, s["h"].shape[1]
    xhat = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (g - xhat * ((g * xhat).sum(1, keepdim=True) / d))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(t), "dweight": (dy * xhat).sum(0).to(s["weight"].dtype)}


def _positions(s):
    """(key minus query position, what is left by the masks or None), [batch or 1, q, k] each."""
    c, dev = s["case"], s["table"].device
    at = torch.as_tensor(s["q_offset"], device=dev).reshape(-1, 1) + torch.arange(c["q"], device=dev)
    at, key = at[:, :, None], torch.arange(c["k"], device=dev)
    rel, seen = key - at, None
    if c["causal"]:
        seen = rel <= 0
    if s["lengths"] is not None:
        n = s["lengths"][:, None, None]
        inside = (at < n) & (key < n)
        seen = inside if seen is None else seen & inside
    return rel, seen


def _buckets(c, rel):
    """Bucket of each relative position: exact for near ones, by the logarithm for far ones."""
    n, first = c["buckets"], 0
    far = (-rel).clamp_min(0)
    if c["two_sided"]:
        n = n // 2
        first, far = n * (rel > 0), rel.abs()
    near = n // 2
    # 64 bits and 1e-9 keep a distance that lies on a border above it
    step = torch.log(far.clamp_min(1).double() / near) * ((n - near) / math.log(c["distance"] / near))
    log = (near + torch.floor(step + 1e-9).long()).clamp_max(n - 1)
    return first + torch.where(far < near, far, log)


def _bias(s):
    c = s["case"]
    rel, seen = _positions(s)
    bias = s["table"].float().t()[:, _buckets(c, rel)].transpose(0, 1)      # [batch or 1, h, q, k]
    if s["scores"] is not None:
        bias = s["scores"].float() + bias
    if seen is not None:
        bias = bias.masked_fill(~seen[:, None], -math.inf)
    return bias.to(s["table"].dtype)


def _bias_backward(s):
    c, dout = s["case"], s["dout"].float()
    rel, seen = _positions(s)
    if seen is not None:
        dout = dout.masked_fill(~seen[:, None], 0.0)
    b, h, q, k = dout.shape
    # each row one place further to the right than the row below it: a diagonal becomes a column
    dout = torch.nn.functional.pad(dout.flip(2), (0, q)).view(b, h, -1)[:, :, :q * (k + q - 1)]
    diagonals = dout.reshape(b, h, q, k + q - 1).sum((0, 2), dtype=torch.float64)
    rel = torch.arange(k + q - 1, device=dout.device) - (q - 1) - c["k"] + q      # q_offset = k - q
    hot = _buckets(c, rel)[:, None] == torch.arange(c["buckets"], device=dout.device)
    return (hot.double().t() @ diagonals.t()).to(s["table"].dtype)


def _logp(s):
    c = s["case"]
    z = s["logits"].float() * c["scale"]
    rows, vocab = z.shape
    m = z.amax(1, keepdim=True)
    z -= m
    e = z.exp()
    total = e.sum(1, keepdim=True)
    log_total = total.log()
    entropy = (log_total - (e * z).sum(1, keepdim=True) / total)[:, 0]
    scored = s["targets"] >= 0
    at = torch.where(scored, s["targets"], 0)[:, None]
    logp = torch.where(scored, (z.gather(1, at) - log_total)[:, 0], 0.0)
    out = {"logp": logp, "entropy": entropy, "lse": (m + log_total)[:, 0]}
    if c["top"]:
        # order by value, then by the lower index: one whole number for both
        i = (s["logits"].float() + 0.0).view(torch.int32)      # -0 counts as 0
        i = torch.where(i < 0, i ^ 0x7FFFFFFF, i).long()
        key = (i << 32) + (vocab - 1 - torch.arange(vocab, device=z.device))
        ids = vocab - 1 - (key.topk(c["top"], 1).values & 0xFFFFFFFF)
        out.update(top_logp=z.gather(1, ids) - log_total, top_ids=ids)
    return out


def _logp_backward(s, lse, entropy):
    c = s["case"]
    log = (s["logits"].float() * c["scale"]).sub_(lse[:, None])
    scored = s["targets"] >= 0
    dlogp = torch.where(scored, s["dlogp"], 0.0)
    p = log.exp()
    log.add_(entropy[:, None]).mul_(s["dentropy"][:, None]).add_(dlogp[:, None])
    d = p.mul_(log).neg_()
    rows = torch.arange(d.shape[0], device=d.device)
    d[rows, torch.where(scored, s["targets"], 0)] += dlogp
    return d.mul_(c["scale"]).to(s["logits"].dtype)


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _norm(s)
    if op == "norm_backward":
        return _norm_backward(s)
    if op == "bias":
        return {"out": _bias(s)}
    if op == "bias_backward":
        return {"dtable": _bias_backward(s)}
    if op == "bias_train":
        return {"out": _bias(s), "dtable": _bias_backward(s)}
    if op == "logp":
        return _logp(s)
    if op == "logp_backward":
        return {"dlogits": _logp_backward(s, s["lse"], s["entropy"])}
    out = _logp(s)
    return {**out, "dlogits": _logp_backward(s, out["lse"], out["entropy"])}


# ------------------------------------------------------------------ the library's calls

def _own(s):
    from scan_fixed_order_amd import det

    c = s["case"]
    op, out = c["op"], {}
    if op == "norm":
        r = det.det_rms_norm(s["x"], s["weight"], eps=_EPS, residual=s["residual"],
                             quant=torch.float8_e4m3fn if c["bits8"] else None, group=c["group"])
        out = {"y": r.y}
        if s["residual"] is not None:
            out["h"] = r.h
        if c["bits8"]:
            out["scales"] = r.scales
    elif op == "norm_backward":
        out["dx"], out["dweight"] = det.det_rms_norm_backward(s["dy"], s["h"], s["weight"],
                                                              s["rstd"], dh=s["dh"])
    elif op.startswith("bias"):
        how = {"max_distance": c["distance"], "bidirectional": c["two_sided"],
               "causal": c["causal"], "q_offset": s["q_offset"], "lengths": s["lengths"]}
        if op != "bias_backward":
            out["out"] = det.det_relative_bias(s["table"], c["q"], c["k"], scores=s["scores"], **how)
        if op != "bias":
            out["dtable"] = det.det_relative_bias_backward(s["dout"], c["buckets"], **how)
    else:
        lse, entropy = s.get("lse"), s.get("entropy")
        if op != "logp_backward":
            r = det.det_token_logprobs(s["logits"], s["targets"], scale=c["scale"], top=c["top"])
            out = {"logp": r.logp, "entropy": r.entropy, "lse": r.lse}
            if c["top"]:
                out.update(top_logp=r.top_logp, top_ids=r.top_ids)
            lse, entropy = r.lse, r.entropy
        if op != "logp":
            out["dlogits"] = det.det_token_logprobs_backward(
                s["logits"], s["targets"], lse, s["dlogp"], entropy=entropy,
                dentropy=s["dentropy"], scale=c["scale"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, e, op = case, _BYTES[case["type"]], case["op"]
    if op.startswith("norm"):
        n, d, rows = c["rows"] * c["d"], c["d"], c["rows"]
        if op == "norm":
            groups = rows * -(-d // (c["group"] or d)) if c["bits8"] else 0
            read = n * e * (2 if c["residual"] else 1) + d * e
            write = n * (1 if c["bits8"] else e) + (n * e if c["residual"] else 0) + 4 * groups
            return {"bytes": read + write, "flops": n * 6}
        return {"bytes": n * e * (4 if c["residual"] else 3) + 4 * rows + 2 * d * e, "flops": n * 10}
    if op.startswith("bias"):
        maps = c["batch"] if c["scores"] or (c["ragged"]) else 1
        q, k = c["q"], c["k"]
        full = c["heads"] * q * k
        # of the gradient, what the causal mask leaves (a ragged batch: three quarters of its keys)
        first = k - q
        left = sum(range(first + 1, k + 1)) / (q * k) if c["causal"] else 1.0
        left *= 0.75 if c["ragged"] else 1.0
        table = c["buckets"] * c["heads"] * e
        bytes_, flops = 0, 0
        if op != "bias_backward":
            bytes_ += maps * full * e + table + (left * maps * full * e if c["scores"] else 0)
            flops += maps * full
        if op != "bias":
            bytes_ += left * c["batch"] * full * e + table
            flops += left * c["batch"] * full
        return {"bytes": bytes_, "flops": flops}
    n, rows = c["rows"] * c["vocab"], c["rows"]
    bytes_, flops = 0, 0
    if op != "logp_backward":
        bytes_ += n * e + rows * (8 + 12 + 12 * c["top"])
        flops += n * 6
    if op != "logp":
        bytes_ += 2 * n * e + rows * (8 + 16)
        flops += n * 8
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_norm(s):
    c = s["case"]
    h = s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + _EPS)
    y = y * s["weight"].double()
    out = {"h": h} if s["residual"] is not None else {}
    if not c["bits8"]:
        return {**out, "y": y}
    group = c["group"] or c["d"]
    parts = [p.abs().amax(1).clamp_min(_TINY) / _E4M3_MAX for p in y.split(group, 1)]
    scales = torch.stack(parts, 1)
    return {**out, "y": y / scales.repeat_interleave(group, 1)[:, :c["d"]], "scales": scales}


def _exact_norm_backward(s):
    h, dy, w, r = s["h"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()[:, None]
    inner = (dy * w * h).sum(1, keepdim=True)
    dx = r * dy * w - h * r ** 3 * inner / h.shape[1]
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {"dx": dx, "dweight": (dy * (h * r)).sum(0)}


def _exact_starts(n, distance):
    """The first distance of each of a side's n buckets, in whole numbers: bucket near + j starts at
    the least a with (a / near) ** (n - near) >= (distance / near) ** j."""
    near, starts, a = n // 2, [], 0
    for j in range(n):
        if j < near:
            a = j
        else:
            a = max(a, near)
            while a ** (n - near) * near ** (j - near) < distance ** (j - near) * near ** (n - near):
                a += 1
        starts.append(a)
    return starts


def _exact_buckets(c, rel):
    n = c["buckets"] // 2 if c["two_sided"] else c["buckets"]
    starts = torch.tensor(_exact_starts(n, c["distance"]), device=rel.device)
    far = rel.abs() if c["two_sided"] else torch.where(rel < 0, -rel, 0)
    side = torch.searchsorted(starts, far, right=True) - 1
    return torch.where(rel > 0, side + n, side) if c["two_sided"] else side


def _exact_maps(s):
    """For each sequence: its buckets [q, k] and the places that the masks leave."""
    c, dev = s["case"], s["table"].device
    several = s["lengths"] is not None or torch.is_tensor(s["q_offset"])
    for b in range(c["batch"] if several or s["scores"] is not None else 1):
        start = s["q_offset"][b] if torch.is_tensor(s["q_offset"]) else s["q_offset"]
        qi = (torch.arange(c["q"], device=dev) + start)[:, None]
        ki = torch.arange(c["k"], device=dev)[None]
        left = torch.ones(c["q"], c["k"], dtype=torch.bool, device=dev)
        if c["causal"]:
            left &= ki <= qi
        if s["lengths"] is not None:
            left &= (ki < s["lengths"][b]) & (qi < s["lengths"][b])
        yield _exact_buckets(c, ki - qi), left


def _exact_bias(s):
    out = []
    for b, (bucket, left) in enumerate(_exact_maps(s)):
        one = s["table"].double().index_select(0, bucket.flatten()).t().reshape(-1, *bucket.shape)
        if s["scores"] is not None:
            one = one + s["scores"][b].double()
        out.append(torch.where(left, one, -math.inf))
    return torch.stack(out)


def _exact_bias_backward(s):
    c, maps = s["case"], list(_exact_maps(s))
    total = torch.zeros(c["buckets"], c["heads"], dtype=torch.float64, device=s["table"].device)
    for b in range(c["batch"]):
        bucket, left = maps[b if len(maps) > 1 else 0]
        g = torch.where(left, s["dout"][b].double(), 0.0)
        for j in range(c["buckets"]):
            total[j] += (g * (bucket == j)).sum((1, 2))
    return total


def _exact_logp(s):
    c = s["case"]
    parts = []
    for z, at in zip(s["logits"].split(256), s["targets"].split(256)):
        z = z.double() * c["scale"]
        lse = torch.logsumexp(z, 1)
        log = z - lse[:, None]
        picked = log.gather(1, at.clamp_min(0)[:, None])[:, 0]
        one = {"logp": torch.where(at < 0, 0.0, picked), "entropy": -(log.exp() * log).sum(1),
               "lse": lse}
        if c["top"]:
            order = z.sort(dim=1, descending=True, stable=True)
            one["top_logp"] = order.values[:, :c["top"]] - lse[:, None]
            one["top_ids"] = order.indices[:, :c["top"]].clone()
        parts.append(one)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_logp_backward(s, lse, entropy):
    c, parts = s["case"], []
    for i in range(0, c["rows"], 512):
        r = slice(i, i + 512)
        log = s["logits"][r].double() * c["scale"] - lse[r].double()[:, None]
        p, scored = log.exp(), (s["targets"][r] >= 0)[:, None]
        hit = torch.zeros_like(p).scatter_(1, s["targets"][r].clamp_min(0)[:, None], 1.0)
        d = torch.where(scored, s["dlogp"][r].double()[:, None], 0.0) * (hit - p)
        d -= s["dentropy"][r].double()[:, None] * p * (log + entropy[r].double()[:, None])
        parts.append(c["scale"] * d)
    return torch.cat(parts)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_backward":
        return _exact_norm_backward(s)
    if op.startswith("bias"):
        out = {}
        if op != "bias_backward":
            out["out"] = _exact_bias(s)
        if op != "bias":
            out["dtable"] = _exact_bias_backward(s)
        return out
    if op == "logp":
        return _exact_logp(s)
    if op == "logp_backward":
        return {"dlogits": _exact_logp_backward(s, s["lse"], s["entropy"])}
    out = _exact_logp(s)
    return {**out, "dlogits": _exact_logp_backward(s, out["lse"], out["entropy"])}
