"""Cases, inputs and plain forms of the gradients around an attention layer: the
attention's backward pass, and the norm of queries and keys for each head with
the rotary positions in the same pass (forward and gradient).

``own`` False: elementary torch operations in 32 bits (angles, and sums over all
tokens, in 64).  ``own`` True: the calls a user makes of this package.
"""
import math

import torch

own = False

PAIRINGS = ("adjacent", "halves")
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# Head dimension -> rotary dimensions of the (time, height, width) axes.
AXES = {128: (16, 56, 56), 64: (16, 24, 24), 32: (8, 12, 12)}
EPS = 1e-6
LARGEST_PAIRS = 24 * 16896 * 16896
LARGEST_VALUES = 119056 * 48 * 128


def listed():
    return [
        # The smallest call: 4 heads of 32, 256 tokens, a gradient of LSE too.
        dict(name="grad 4x256", op="attend", B=1, Hq=4, Hk=4, Nq=256, Nk=256, D=32, mask="none", heads=1,
             causal=False, dlse=True),
        # SD1.5 512^2 UNet self-attention, a batch of two.
        dict(name="grad sd self 4096", op="attend", B=2, Hq=8, Hk=8, Nq=4096, Nk=4096, D=64, mask="none", heads=1,
             causal=False, dlse=False),
        # Its cross-attention to 77 text tokens padded to 80.
        dict(name="grad sd cross 4096x80", op="attend", B=2, Hq=8, Hk=8, Nq=4096, Nk=80, D=64, mask="key", heads=1,
             causal=False, dlse=False),
        # FLUX 1024^2 joint attention.
        dict(name="grad flux 4608", op="attend", B=1, Hq=24, Hk=24, Nq=4608, Nk=4608, D=128, mask="none", heads=1,
             causal=False, dlse=False),
        # The same at 2048^2: the largest.
        dict(name="grad flux 16896", op="attend", B=1, Hq=24, Hk=24, Nq=16896, Nk=16896, D=128, mask="none", heads=1,
             causal=False, dlse=False),
        # Causal training on an odd length, four query heads to each key head.
        dict(name="grad causal 2x4001", op="attend", B=2, Hq=32, Hk=8, Nq=4001, Nk=4001, D=128, mask="none", heads=1,
             causal=True, dlse=False),
        # Sequences packed into one row, each to itself (a boolean mask), some padding rows that see nothing.
        dict(name="grad packed 1777 bool", op="attend", B=2, Hq=12, Hk=12, Nq=1777, Nk=1777, D=64, mask="bool",
             heads=1, causal=False, dlse=False),
        # A bias for each head and pair, added to the scores.
        dict(name="grad bias 1024", op="attend", B=2, Hq=16, Hk=16, Nq=1024, Nk=1024, D=64, mask="add", heads=16,
             causal=False, dlse=False),
        # Queries and keys of one HunyuanVideo 720p layer: 256 text tokens at
        # position zero, then a 33 x 45 x 80 latent grid.
        dict(name="norm rope video 119056", op="norm", B=1, Hq=24, Hk=24, D=128, text=256, t=33, h=45, w=80,
             dtype="bf16", weight="bf16", pairing="adjacent", back=False),
        # FLUX 1024^2: the gradient, back to the token-major projection.
        dict(name="norm rope gradient 4608", op="norm", B=1, Hq=24, Hk=24, D=128, text=512, t=1, h=64, w=64,
             dtype="bf16", weight="fp32", pairing="adjacent", back=True),
        # The gradient at 2048^2 in 32 bits.
        dict(name="norm rope gradient 16896 fp32", op="norm", B=1, Hq=24, Hk=24, D=128, text=512, t=1, h=128, w=128,
             dtype="fp32", weight="fp32", pairing="adjacent", back=True),
        # One new token for each of 16 sequences, shared key heads: a decode step.
        dict(name="norm rope token 16x1", op="norm", B=16, Hq=32, Hk=8, D=64, text=0, t=1, h=1, w=1,
             dtype="fp16", weight="fp16", pairing="halves", back=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    D = rng.choice((32, 64, 128))
    Hk = rng.randint(1, 24)
    if rng.random() < 0.4:
        B = _log(rng, 1, 32)
        n = _log(rng, 1, 16896)
        t, h = rng.choice(((1, 1), (1, _log(rng, 1, 64)), (_log(rng, 1, 16), _log(rng, 1, 32))))
        w = max(1, n // (t * h))
        text = rng.choice((0, 0, rng.randint(1, 512)))
        Hq = Hk * rng.choice((1, 2, 4))
        B = max(1, min(B, LARGEST_VALUES // (2 * (text + t * h * w) * (Hq + Hk) * D)))
        dtype = rng.choice(tuple(DTYPES))
        return dict(op="norm", B=B, Hq=Hq, Hk=Hk, D=D, text=text, t=t, h=h, w=w, dtype=dtype,
                    weight=rng.choice((dtype, "fp32", "none")), pairing=rng.choice(PAIRINGS), back=rng.random() < 0.6)
    Hq = Hk * rng.choice((1, 1, 2, 4, 8))
    B = _log(rng, 1, 8)
    Nq = _log(rng, 1, 16896)
    Nk = Nq if rng.random() < 0.6 else _log(rng, 1, 16896)
    mask = rng.choice(("none", "none", "key", "bool", "add"))
    heads = rng.choice((1, Hq)) if mask in ("bool", "add") else 1
    most = LARGEST_PAIRS // (4 if mask in ("bool", "add") else 2)
    while B * Hq * Nq * Nk > most:
        if B > 1:
            B //= 2
        elif Nq >= Nk:
            Nq //= 2
        else:
            Nk //= 2
    # (with few keys a gradient of LSE too: a row of one key has no other gradient of q)
    dlse = min(Nq, Nk) < 16 or rng.random() < 0.2
    return dict(op="attend", B=B, Hq=Hq, Hk=Hk, Nq=Nq, Nk=Nk, D=D, mask=mask, heads=heads,
                causal=rng.random() < 0.35, dlse=dlse)


def _positions(case, seed):
    grid = torch.cartesian_prod(*(torch.arange(n) for n in (case["t"], case["h"], case["w"])))
    B, text = case["B"], case["text"]
    pos = torch.zeros(B, text + grid.shape[0], 3, dtype=torch.int32)
    pos[:, text:] = grid.to(torch.int32)
    if grid.shape[0] == 1:  # a decode step: each sequence at a place of its own
        pos[:, text:] += torch.randint(0, 200000, (B, 1, 3), generator=torch.Generator().manual_seed(seed),
                                       dtype=torch.int32)
    return pos.cuda()


def _mask(case, g):
    """The mask tensor of a case, or None: fp32 [B, Nk], or bool / fp32 [B, heads, Nq, Nk]."""
    B, heads, Nq, Nk = case["B"], case["heads"], case["Nq"], case["Nk"]
    if case["mask"] == "key":  # valid lengths, -inf behind them
        valid = torch.randint(max(1, Nk // 4), Nk + 1, (B, 1), generator=g, device="cuda")
        return torch.where(torch.arange(Nk, device="cuda") < valid, 0.0, -math.inf)
    if case["mask"] == "bool":  # packed sequences; the last rows are padding and see nothing
        cuts = max(1, min(Nq, Nk) // 300)
        row, key = (torch.arange(n, device="cuda") * cuts // n for n in (Nq, Nk))
        keep = (row[:, None] == key)[None, None].repeat(B, heads, 1, 1)
        keep &= torch.rand(B, heads, 1, Nk, generator=g, device="cuda") < 0.9
        keep[:, :, Nq - Nq // 50:] = False
        return keep
    if case["mask"] == "add":
        m = torch.randn(B, heads, Nq, Nk, generator=g, device="cuda")
        return m.masked_fill_(torch.rand(B, heads, 1, Nk, generator=g, device="cuda") < 0.1, -math.inf)
    return None


def _add_mask(t, s):
    """Scores t [B, Hk, g, Nq, Nk] with the case's mask, in place."""
    m = s["m"]
    if s["mask"] == "key":
        t += m[:, None, None, None]
    elif s["mask"] != "none":
        m = m.unsqueeze(1) if s["heads"] == 1 else m.view(m.shape[0], t.shape[1], t.shape[2], *m.shape[2:])
        t = t.masked_fill_(~m, -math.inf) if s["mask"] == "bool" else t.add_(m)
    if s["causal"]:
        row, key = (torch.arange(n, device=t.device) for n in t.shape[3:])
        t.masked_fill_(key > row[:, None], -math.inf)
    return t


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    B, Hq, Hk, D = case["B"], case["Hq"], case["Hk"], case["D"]
    if case["op"] == "norm":
        dtype = DTYPES[case["dtype"]]
        s["pos"] = _positions(case, seed)
        N = s["pos"].shape[1]
        s["dims"], s["theta"] = AXES[D], 10000.0
        # slices of the token-major projection of q, k and v; rows of unequal size
        x = torch.randn(B, N, Hq + 2 * Hk, D, generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(B, N, 1, 1, generator=g, device="cuda"))
        x = x.to(dtype)
        s["q"], s["k"] = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
        weights = [1.0 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
        s["wq"], s["wk"] = ((None, None) if case["weight"] == "none" else
                            (w.to(DTYPES[case["weight"]]) for w in weights))
        if case["back"]:  # gradients as the attention leaves them, head-major
            s["dq"] = torch.randn(B, Hq, N, D, generator=g, device="cuda").to(dtype)
            s["dk"] = torch.randn(B, Hk, N, D, generator=g, device="cuda").to(dtype)
        return s
    Nq, Nk = case["Nq"], case["Nk"]
    s["q"] = torch.randn(B, Hq, Nq, D, generator=g, device="cuda").to(torch.bfloat16)
    s["k"], s["v"] = (torch.randn(B, Hk, Nk, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    # the gradient of O, as the output projection leaves it: token-major
    s["dout"] = torch.randn(B, Nq, Hq, D, generator=g, device="cuda").to(torch.bfloat16).transpose(1, 2)
    s["dlse_"] = torch.randn(B, Hq, Nq, generator=g, device="cuda") if case["dlse"] else None
    s["m"] = _mask(case, g)
    s["scale"] = 1.0 / math.sqrt(D)
    # O and LSE, which the forward left
    s["out"] = torch.empty(B, Hq, Nq, D, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(B, Hq, Nq, device="cuda")
    for b in range(B):
        for h in range(Hq):
            at = h * Hk // Hq
            t = (s["q"][b, h].float() @ s["k"][b, at].float().T * s["scale"])[None, None, None]
            one = dict(s, heads=1)
            if case["mask"] == "key":
                one["m"] = s["m"][b:b + 1]
            elif case["mask"] != "none":
                hm = h if case["heads"] > 1 else 0
                one["m"] = s["m"][b:b + 1, hm:hm + 1]
            t = _add_mask(t, one)[0, 0, 0]
            m = t.amax(-1, keepdim=True).clamp(min=-1e30)
            p = t.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            s["out"][b, h] = (p @ s["v"][b, at].float() / l.clamp(min=1e-30)).to(torch.bfloat16)
            s["lse"][b, h] = (m + torch.log(l))[:, 0]
    return s


def _turn(x, pos, dims, theta, pairing, back):
    """x (32 bits) turned by its positions, or back."""
    freq = torch.cat([theta ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d) for d in dims])
    axis = torch.cat([torch.full((d // 2,), a, device=x.device) for a, d in enumerate(dims)])
    angle = torch.remainder(pos.double()[:, None, :, axis] * freq, 2 * math.pi)
    cos, sin = angle.cos().float(), angle.sin().float()
    if back:
        sin = -sin
    D = x.shape[-1]
    a, b = (x[..., 0::2], x[..., 1::2]) if pairing == "adjacent" else (x[..., :D // 2], x[..., D // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.stack((a, b), -1).flatten(-2) if pairing == "adjacent" else torch.cat((a, b), -1)


def _norm(x, w, s):
    """The rows' norm, the weight and the rotation."""
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    y = y if w is None else y * w.float()
    return _turn(y, s["pos"], s["dims"], s["theta"], s["pairing"], False).to(x.dtype)


def _norm_back(dy, x, w, s):
    """Gradients of the same with respect to x and the weight."""
    g = _turn(dy.float(), s["pos"], s["dims"], s["theta"], s["pairing"], True)
    y = x.float()
    r = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    n = y * r
    dw = None if w is None else (g * n).sum((0, 1, 2), dtype=torch.float64).float()
    g = g if w is None else g * w.float()
    return (r * (g - n * (g * n).mean(-1, keepdim=True))).to(x.dtype), dw


def run(s):
    if own:
        import unet_fa_fwd_gb300 as fa
    if s["op"] == "norm":
        if own:
            axes = fa.RopeAxes(s["dims"], s["theta"])
            if s["back"]:
                got = fa.norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["pos"], axes, s["wq"], s["wk"], eps=EPS,
                                       pairing=s["pairing"], token_major=True)
                return got if s["wq"] is not None else got[:2]
            return fa.norm_rope(s["q"], s["k"], s["pos"], axes, s["wq"], s["wk"], eps=EPS, pairing=s["pairing"])
        if s["back"]:
            (dq, dwq), (dk, dwk) = (_norm_back(s[d], s[x], s[w], s) for d, x, w in (("dq", "q", "wq"),
                                                                                  ("dk", "k", "wk")))
            return (dq, dk) if dwq is None else (dq, dk, dwq, dwk)
        return _norm(s["q"], s["wq"], s), _norm(s["k"], s["wk"], s)
    if own:
        masks = {"key": dict(key_mask=s["m"]), "none": {}}.get(s["mask"], dict(full_mask=s["m"]))
        return fa.bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], causal=s["causal"], scale=s["scale"],
                      dlse=s["dlse_"], **masks)
    B, Hq, Nq, D = s["q"].shape
    Hk, Nk = s["Hk"], s["Nk"]
    g = Hq // Hk
    q, dout = (s[n].float().reshape(B, Hk, g * Nq, D) for n in ("q", "dout"))
    k, v = s["k"].float(), s["v"].float()
    t = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    _add_mask(t.view(B, Hk, g, Nq, Nk), s)
    lse = torch.where(torch.isinf(s["lse"]), math.inf, s["lse"]).view(B, Hk, g * Nq, 1)  # a row without keys: P = 0
    p = t.sub_(lse).exp_()
    dv = torch.matmul(p.transpose(2, 3), dout)
    delta = (dout * s["out"].float().view(B, Hk, g * Nq, D)).sum(-1, keepdim=True)
    if s["dlse_"] is not None:
        delta = delta - s["dlse_"].view(B, Hk, g * Nq, 1)
    ds = torch.matmul(dout, v.transpose(2, 3)).sub_(delta).mul_(p)
    dq = torch.matmul(ds, k).mul_(s["scale"])
    dk = torch.matmul(ds.transpose(2, 3), q).mul_(s["scale"])
    return tuple(x.to(torch.bfloat16) for x in (dq.view(B, Hq, Nq, D), dk, dv))


def work(case):
    B, Hq, Hk, D = case["B"], case["Hq"], case["Hk"], case["D"]
    if case["op"] == "norm":
        n = B * (case["text"] + case["t"] * case["h"] * case["w"])
        width = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        values = n * (Hq + Hk) * D
        if case["back"]:
            return dict(bytes=3 * width * values + 12 * n, flops=14 * values)
        return dict(bytes=2 * width * values + 12 * n, flops=7 * values)
    Nq, Nk = case["Nq"], case["Nk"]
    pairs = B * Hq * (sum(min(i + 1, Nk) for i in range(Nq)) if case["causal"] else Nq * Nk)
    mask = {"none": 0, "key": 4 * B * Nk}.get(case["mask"],
                                              B * case["heads"] * Nq * Nk * (1 if case["mask"] == "bool" else 4))
    return dict(bytes=B * D * 2 * (4 * Hq * Nq + 4 * Hk * Nk) + 4 * B * Hq * Nq * (2 if case["dlse"] else 1) + mask,
                flops=10 * D * pairs)


def exact(case, seed):
    s = prepare(case, seed)
    B, Hq, Hk, D = case["B"], case["Hq"], case["Hk"], case["D"]
    if case["op"] == "norm":
        half = D // 2
        phase = [s["pos"][:, :, a].double() * s["theta"] ** (-2.0 * j / d)
                 for a, d in enumerate(s["dims"]) for j in range(d // 2)]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.stack(phase, -1))  # [B, N, half]
        place = (lambda z: torch.view_as_real(z).flatten(-2)) if case["pairing"] == "adjacent" else (
            lambda z: torch.cat((z.real, z.imag), -1))
        pairs = (lambda y: torch.view_as_complex(y.unflatten(-1, (half, 2)).contiguous())) if (
            case["pairing"] == "adjacent") else (lambda y: torch.complex(y[..., :half].contiguous(),
                                                                         y[..., half:].contiguous()))
        got, dws = [], []
        for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
            w64 = torch.ones(D, dtype=torch.float64, device="cuda") if w is None else w.double()
            out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            dw = torch.zeros(D, dtype=torch.float64, device="cuda")
            for h in range(x.shape[1]):
                y = x[:, h].double()
                size = (torch.einsum("bnd,bnd->bn", y, y) / D + EPS).sqrt()[..., None]
                if dy is None:
                    out[:, h] = place(pairs(y / size * w64) * turn)
                    continue
                g = place(pairs(dy[:, h].double()) * turn.conj())
                dw += torch.einsum("bnd,bnd->d", g, y / size)
                along = torch.einsum("bnd,bnd->bn", g * w64, y)[..., None]
                out[:, h] = g * w64 / size - y * along / (D * size ** 3)
            got.append(out)
            dws.append(dw)
        return got + dws if case["back"] and s["wq"] is not None else got
    Nq, Nk = case["Nq"], case["Nk"]
    dq = torch.empty(B, Hq, Nq, D, dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros(B, Hk, Nk, D, dtype=torch.float64, device="cuda") for _ in range(2))
    below = torch.ones(Nq, Nk, dtype=torch.bool, device="cuda").tril() if case["causal"] else None
    for b in range(B):
        for h in range(Hq):
            at = h // (Hq // Hk)
            q, k, v, do = (x.double() for x in (s["q"][b, h], s["k"][b, at], s["v"][b, at], s["dout"][b, h]))
            t = torch.einsum("id,jd->ij", q, k) * s["scale"]
            keep = torch.ones_like(t, dtype=torch.bool) if below is None else below.clone()
            if case["mask"] == "key":
                t = t + s["m"][b].double()
            elif case["mask"] == "add":
                t = t + s["m"][b, h if case["heads"] > 1 else 0].double()
            elif case["mask"] == "bool":
                keep &= s["m"][b, h if case["heads"] > 1 else 0]
            lse = s["lse"][b, h].double()
            p = torch.where(keep & torch.isfinite(lse)[:, None], torch.exp(t - lse[:, None]), 0.0)
            grow = torch.einsum("id,id->i", do, s["out"][b, h].double())
            if s["dlse_"] is not None:
                grow = grow - s["dlse_"][b, h].double()
            ds = p * (torch.einsum("id,jd->ij", do, v) - grow[:, None])
            dv[b, at] += torch.einsum("ij,id->jd", p, do)
            dk[b, at] += torch.einsum("ij,id->jd", ds, q) * s["scale"]
            dq[b, h] = torch.einsum("ij,jd->id", ds, k) * s["scale"]
    return [dq, dk, dv]
