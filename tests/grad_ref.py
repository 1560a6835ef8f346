"""64-bit definitions of the norm with rotary positions, its gradient and the
attention's gradient, for the tests (torch, on whatever device the inputs are)."""
import math

import torch

from . import cache_ref


def pair_size(x, pairing):
    """|x0| + |x1| of each element's pair: what bounds a rotated pair."""
    a, D = x.abs(), x.shape[-1]
    if pairing == "adjacent":
        return a.unflatten(-1, (D // 2, 2)).sum(-1).repeat_interleave(2, -1)
    return (a[..., :D // 2] + a[..., D // 2:]).repeat(1, 1, 1, 2)


def norm(x, w, eps):
    """(x / sqrt(mean(x^2) + eps), that times w, 1 / the root), in 64 bits."""
    x = x.double()
    r = 1.0 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return x * r, x * r * (1.0 if w is None else w.double()), r


def norm_rope(x, w, eps, pos, dims, pairing, **kw):
    return cache_ref.rope(norm(x, w, eps)[1], pos, dims, pairing=pairing, **kw)


def norm_rope_bwd(dy, x, w, eps, pos, dims, pairing, **kw):
    """(dx, dw, bounds of their terms' sizes), in 64 bits."""
    n, _, r = norm(x, w, eps)
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
    g = cache_ref.rope(dy, pos, dims, pairing=pairing, inverse=True, **kw)
    size = pair_size(dy.double(), pairing)
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    dx_size = r * (size * w.abs() + n.abs() * (size * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, (g * n).sum((0, 1, 2)), dx_size, (size * n.abs()).sum((0, 1, 2))


def scores(q, k, scale, key_mask=None, full_mask=None, causal=False):
    """Scaled, masked scores [B, Hq, Nq, Nk] in 64 bits; -inf where a pair is excluded."""
    g = q.shape[1] // k.shape[1]
    t = q.double() @ k.double().repeat_interleave(g, 1).transpose(2, 3) * scale
    if key_mask is not None:
        t = t + key_mask.double()[:, None, None]
    if full_mask is not None:
        t = t.masked_fill(full_mask == 0, -math.inf) if full_mask.dtype in (torch.bool, torch.uint8) else (
            t + full_mask.double())
    if causal:
        row, key = (torch.arange(n, device=t.device) for n in t.shape[2:])
        t = t.masked_fill(key > row[:, None], -math.inf)
    return t


def attend(q, k, v, scale, **masks):
    """(O, LSE) in 64 bits; rows without a key give zeros and -inf."""
    t = scores(q, k, scale, **masks)
    lse = torch.logsumexp(t, -1)
    p = torch.where(torch.isneginf(t), 0.0, torch.exp(t - lse[..., None]))
    return p @ v.double().repeat_interleave(q.shape[1] // k.shape[1], 1), lse


def attend_bwd(dout, q, k, v, out, lse, scale, dlse=None, **masks):
    """(dq, dk, dv) in 64 bits from what the forward left, and for each the sum of
    the sizes of its terms (what errors of the probabilities scale with)."""
    g = q.shape[1] // k.shape[1]
    t = scores(q, k, scale, **masks)
    p = torch.where(torch.isneginf(t), 0.0, torch.exp(t - lse.double()[..., None]))
    do, kk, vv = dout.double(), k.double().repeat_interleave(g, 1), v.double().repeat_interleave(g, 1)
    delta = (do * out.double()).sum(-1)
    delta_size = (do * out.double()).abs().sum(-1)
    if dlse is not None:
        delta, delta_size = delta - dlse.double(), delta_size + dlse.double().abs()
    ds = p * (do @ vv.transpose(2, 3) - delta[..., None])
    # what fp32 sums in dP and delta can be off by, relative to 2^-24 a term
    ds_size = p * (do.abs() @ vv.abs().transpose(2, 3) + delta_size[..., None])

    def join(x):  # heads that share a key head
        return x.unflatten(1, (k.shape[1], g)).sum(2)

    T = lambda x: x.transpose(2, 3)  # noqa: E731
    got = (ds @ kk * scale, join(T(ds) @ q.double()) * scale, join(T(p) @ do))
    size = (ds.abs() @ kk.abs() * abs(scale), join(T(ds.abs()) @ q.double().abs()) * abs(scale),
            join(T(p) @ do.abs()))
    fine = (ds_size @ kk.abs() * abs(scale), join(T(ds_size) @ q.double().abs()) * abs(scale), size[2])
    return got, size, fine
