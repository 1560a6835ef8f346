"""64-bit definitions of the rotary positions, the e4m3 cache and the attention
to it, for the tests (torch, on whatever device the inputs are)."""
import math

import torch

EXP_MIN, EXP_MAX = -117, 119


def rope(x, pos, dims, theta=10000.0, scale=1.0, pairing="adjacent", inverse=False):
    """x [B, H, N, D] turned by pos [B, N, A] (or [N, A]), in 64 bits."""
    if pos.dim() == 2:
        pos = pos.expand(x.shape[0], *pos.shape)
    one = lambda v, a: float(v[a]) if isinstance(v, (tuple, list)) else float(v)  # noqa: E731
    angle = torch.cat([pos[:, :, a:a + 1].double() * one(scale, a)
                       * one(theta, a) ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d)
                       for a, d in enumerate(dims)], -1)[:, None]
    c, s = angle.cos(), angle.sin() * (-1 if inverse else 1)
    x = x.double()
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if pairing == "adjacent" else (x[..., :half], x[..., half:])
    y = torch.empty_like(x)
    if pairing == "adjacent":
        y[..., 0::2], y[..., 1::2] = a * c - b * s, a * s + b * c
    else:
        y[..., :half], y[..., half:] = a * c - b * s, a * s + b * c
    return y


def e4m3(x):
    """x (64 bits) to the nearest e4m3 value, ties to even, saturating at 448."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -9))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def scale_of(amax):
    """Least power of two s in [2^-117, 2^119] with amax <= 448 s (elementwise, 64 bits)."""
    e = torch.ceil(torch.log2(amax.clamp(min=448.0 * 2.0 ** EXP_MIN) / 448.0))
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
    return torch.exp2(e.clamp(EXP_MIN, EXP_MAX))


def quantised(x, page, start=0):
    """Values that a cache holds for x [H, N, D] written in one call at ``start`` of an empty
    sequence: (values, scale of each token [H, N])."""
    x = x.double()
    N = x.shape[1]
    group = (torch.arange(N, device=x.device) + start) // page
    s = torch.empty(x.shape[0], N, dtype=torch.float64, device=x.device)
    for g in group.unique().tolist():
        at = group == g
        s[:, at] = scale_of(x[:, at].abs().amax((1, 2)))[:, None]
    return e4m3(x / s[..., None]) * s[..., None], s


def weight(v, page, tile):
    """|v| times the ratio of the largest scale among the pages of a token's 128-token tile (or of the
    whole sequence) to its own page's: v [H, L, D].  (The scales are taken from what the cache holds, whose largest element may
    have been rounded down past a power of two: the ratio is within a factor of 2.)"""
    H, L, D = v.shape
    pad = torch.zeros(H, -(-L // 128) * 128, D, dtype=v.dtype, device=v.device)
    pad[:, :L] = v.nan_to_num(0.0)
    s = scale_of(pad.abs().view(H, -1, page, D).amax((2, 3)))  # [H, pages]
    most = s.view(H, -1, 128 // page).amax(2).repeat_interleave(128 // page, 1) if tile else s.amax(1, keepdim=True)
    return (pad.abs() * (most / s).repeat_interleave(page, 1)[..., None])[:, :L]


def attend(q, k, v, scale, causal=False, q_start=None):
    """One sequence: q [Hq, Nq, D], k, v [Hk, L, D] in 64 bits.  Returns O, LSE, the mean of |v|
    under each row's probabilities, and over a row's keys the largest sum_d |q k| |scale| and
    max |q| sum_d |k| |scale|."""
    Hq, Nq, D = q.shape
    Hk, L = k.shape[:2]
    q = q.double()
    k, v = (x.double().repeat_interleave(Hq // Hk, 0) for x in (k, v))
    seen = torch.ones(Nq, L, dtype=torch.bool, device=q.device)
    if causal:
        first = L - Nq if q_start is None else q_start
        seen = torch.arange(L, device=q.device) <= first + torch.arange(Nq, device=q.device)[:, None]
    if L == 0 or not seen.any():
        z = torch.zeros(Hq, Nq, D, dtype=torch.float64, device=q.device)
        return z, torch.full((Hq, Nq), -math.inf, dtype=torch.float64, device=q.device), z, z[..., 0], z[..., 0]
    t = torch.where(seen, q @ k.transpose(1, 2) * scale, -math.inf)
    lse = torch.logsumexp(t, -1)
    p = torch.where(seen, torch.exp(t - lse[..., None]), 0.0).nan_to_num(0.0)
    size = (q.abs() @ k.abs().transpose(1, 2) * abs(scale) * seen).amax(-1)
    spread = q.abs().amax(-1) * abs(scale) * k.abs().sum(-1).amax(-1)[:, None]
    return p @ v, lse, p @ v.abs(), size, spread
