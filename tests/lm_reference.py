"""Plain 64-bit statements of the language-model operators, on whatever device the inputs are, and
the step sizes that the tests' tolerances count.  They share no code with the library."""
import math
from fractions import Fraction

import torch

TYPES = [torch.float32, torch.float16, torch.bfloat16]
IDS = ["f32", "f16", "bf16"]
U32 = 2.0 ** -24          # half a step of f32, relative


def half(t):
    """Half a step of a type, relative to the value."""
    return torch.finfo(t).eps / 2


def floor_of(t):
    """Half a step among a type's subnormals: what a rounding is off by at least."""
    return {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -127}[t]


def randn(shape, t, dev, seed, scale=1.0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev) * scale).to(t)


def same_bits(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(
        a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))


def norm(x, weight, eps, residual=None):
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = (h.square().mean(-1) + eps).rsqrt()
    return h, rstd, h * rstd[..., None] * weight.double()


def norm_backward(dy, h, weight, rstd, dh=None):
    dy, h, w, r = dy.double(), h.double(), weight.double(), rstd.double()[..., None]
    xhat = h * r
    g = dy * w
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy * xhat).flatten(0, -2).sum(0)


def bucket(r, buckets, distance, two_sided):
    """Bucket of one relative position, in whole numbers."""
    n = buckets // 2 if two_sided else buckets
    first = n if two_sided and r > 0 else 0
    a = abs(r) if two_sided else max(-r, 0)
    near = n // 2
    if a < near:
        return first + a
    power, j = n - near, 0
    # the largest j with (a / near)^power >= (distance / near)^j
    while j + 1 < power and Fraction(a, near) ** power >= Fraction(distance, near) ** (j + 1):
        j += 1
    return first + near + j


def bias_maps(batch, q, k, buckets, distance, two_sided, causal, offsets, lengths, dev):
    """(bucket, unmasked), [batch, q, k]"""
    offsets = [offsets] * batch if isinstance(offsets, int) else offsets
    seen = {}
    bk = torch.zeros(batch, q, k, dtype=torch.int64)
    left = torch.ones(batch, q, k, dtype=torch.bool)
    i, j = torch.arange(q)[:, None], torch.arange(k)[None]
    for b in range(batch):
        rel = j - i - offsets[b]
        for r in range(-(q - 1) - offsets[b], k - offsets[b]):
            if r not in seen:
                seen[r] = bucket(r, buckets, distance, two_sided)
        low = -(q - 1) - offsets[b]
        line = torch.tensor([seen[low + n] for n in range(q + k - 1)])
        bk[b] = line[rel - low]
        if causal:
            left[b] &= rel <= 0
        if lengths is not None:
            left[b] &= (j < lengths[b]) & (i + offsets[b] < lengths[b])
    return bk.to(dev), left.to(dev)


def bias(table, maps, scores=None):
    bk, left = maps
    out = table.double().t()[:, bk].transpose(0, 1)
    if scores is not None:
        out = out + scores.double()
    return torch.where(left[:, None], out, -math.inf)


def bias_backward(dout, maps, buckets):
    """(dtable, the sums of the magnitudes, dscores)"""
    bk, left = maps
    g = torch.where(left[:, None], dout.double(), 0.0)
    flat, at = g.transpose(0, 1).flatten(1), bk.flatten()
    total = torch.zeros(dout.shape[1], buckets, dtype=torch.float64, device=dout.device)
    sizes = torch.zeros_like(total)
    for b in range(buckets):
        sel = at == b
        total[:, b] = flat[:, sel].sum(1)
        sizes[:, b] = flat[:, sel].abs().sum(1)
    return total.t(), sizes.t(), g


def logprobs(logits, targets, scale):
    """(logp, entropy, lse, log p)"""
    z = logits.double() * scale
    # against the largest first: lse of a row of lowest values has no digits left for log(sum)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    log_sum = (z - m).exp().sum(-1, keepdim=True).log()
    lse = (m + log_sum)[..., 0]
    log = (z - m) - log_sum
    p = log.exp()
    entropy = -torch.where(p > 0, p * log, 0.0).sum(-1)
    ok = (targets >= 0) & (targets < logits.shape[-1])
    at = torch.where(ok, targets, 0)
    return torch.where(ok, log.gather(-1, at[..., None])[..., 0], 0.0), entropy, lse, log


def top_ids(logits, top):
    v = logits.double() + 0.0
    return v.sort(dim=-1, descending=True, stable=True).indices[..., :top]


def logprobs_backward(log, targets, entropy, dlogp, dentropy, scale):
    p = log.exp()
    ok = (targets >= 0) & (targets < log.shape[-1])
    d = torch.where(ok, dlogp.double(), 0.0)
    hit = torch.zeros_like(p).scatter_(-1, torch.where(ok, targets, 0)[..., None], 1.0)
    g = d[..., None] * (hit - p)
    if dentropy is not None:
        term = torch.where(p > 0, p * (log + entropy[..., None]), 0.0)
        g = g - dentropy.double()[..., None] * term
    return scale * g
