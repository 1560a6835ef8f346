"""Cases, inputs and plain forms of the operators around a cached attention:
rotary positions over several axes (forward and gradient), a paged key/value
cache held in e4m3 with a power-of-two scale for each page and head (written
and read back), and the attention that reads it.

``own`` False: elementary torch operations in 32 bits (angles in 64).  ``own``
True: the calls a user makes of this package.
"""
import math

import torch

own = False

PAIRINGS = ("adjacent", "halves")
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# Head dimension -> rotary dimensions of the (time, height, width) axes.
AXES = {128: (16, 56, 56), 64: (16, 24, 24), 32: (8, 12, 12)}
E4M3_MAX = 448.0
SCALE_EXP_MIN, SCALE_EXP_MAX = -117, 119


def listed():
    return [
        # Queries and keys of one HunyuanVideo 720p layer: 256 text tokens at
        # position zero, then a 33 x 45 x 80 latent grid.
        dict(name="rope video 119056", op="rope", B=1, Hq=24, Hk=24, D=128, text=256, t=33, h=45, w=80,
             dtype="bf16", pairing="adjacent", back=False),
        # FLUX 1024^2 joint attention, from the token-major projection.
        dict(name="rope image 4608", op="rope", B=1, Hq=24, Hk=24, D=128, text=512, t=1, h=64, w=64,
             dtype="bf16", pairing="adjacent", back=False),
        # The gradient of the same at 2048^2, in 32 bits, back to token-major.
        dict(name="rope gradient 16896 fp32", op="rope", B=1, Hq=24, Hk=24, D=128, text=512, t=1, h=128, w=128,
             dtype="fp32", pairing="adjacent", back=True),
        # One new token for each of 16 sequences, shared key heads: a decode step.
        dict(name="rope token 16x1", op="rope", B=16, Hq=32, Hk=8, D=64, text=0, t=1, h=1, w=1,
             dtype="fp16", pairing="halves", back=False),
        # Three latent frames of 45 x 80 tokens added to a video's cache.
        dict(name="cache chunk 10800", op="cache", B=1, Hk=24, D=128, page=128, start=10800, N=10800, ragged=False),
        # A ragged batch of prompts, odd lengths, small pages.
        dict(name="cache ragged 7x997", op="cache", B=7, Hk=8, D=64, page=32, start=301, N=997, ragged=True),
        # One token for each of 64 sequences: a decode step.
        dict(name="cache token 64x1", op="cache", B=64, Hk=8, D=128, page=64, start=4095, N=1, ragged=True),
        # The smallest call: one sequence, one row, 77 text tokens.
        dict(name="attend 1x77", op="attend", B=1, Hq=8, Hk=8, D=64, page=32, L=77, Nq=1, causal=False, ragged=False),
        # A ragged decode batch with four query heads to each key head.
        dict(name="attend decode 64x8192", op="attend", B=64, Hq=32, Hk=8, D=128, page=64, L=8192, Nq=1,
             causal=True, ragged=True),
        # One query against the cache of a whole 720p video.
        dict(name="attend decode 1x119056", op="attend", B=1, Hq=24, Hk=24, D=128, page=128, L=119056, Nq=1,
             causal=False, ragged=False),
        # A few rows for each sequence (drafted tokens checked at once).
        dict(name="attend draft 8x5x4111", op="attend", B=8, Hq=16, Hk=4, D=64, page=32, L=4111, Nq=5,
             causal=True, ragged=True),
        # A chunk of new tokens attends to itself and to everything cached.
        dict(name="attend chunk 2048x16896", op="attend", B=1, Hq=24, Hk=24, D=128, page=128, L=16896, Nq=2048,
             causal=True, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    D = rng.choice((32, 64, 128))
    Hk = rng.randint(1, 24)
    op = rng.choice(("rope", "cache", "attend", "attend"))
    if op == "rope":
        B = _log(rng, 1, 32)
        n = _log(rng, 1, 16896)
        t, h = rng.choice(((1, 1), (1, _log(rng, 1, 64)), (_log(rng, 1, 16), _log(rng, 1, 32))))
        w = max(1, n // (t * h))
        text = rng.choice((0, 0, rng.randint(1, 512)))
        Hq = Hk * rng.choice((1, 2, 4))
        B = max(1, min(B, 119056 * 24 * 128 // ((text + t * h * w) * (Hq + Hk) * D)))
        return dict(op=op, B=B, Hq=Hq, Hk=Hk, D=D, text=text, t=t, h=h, w=w, dtype=rng.choice(tuple(DTYPES)),
                    pairing=rng.choice(PAIRINGS), back=rng.random() < 0.4)
    page = rng.choice((32, 64, 128))
    B = _log(rng, 1, 64)
    if op == "cache":
        N = 1 if rng.random() < 0.3 else _log(rng, 2, 10800)
        start = rng.choice((0, _log(rng, 1, 10800)))
        B = max(1, min(B, 10800 * 24 * 128 // ((N + page) * Hk * D)))
        return dict(op=op, B=B, Hk=Hk, D=D, page=page, start=start, N=N, ragged=rng.random() < 0.6)
    g = rng.choice((1, 2, 4, 8))
    L = _log(rng, 1, 65536)
    Nq = rng.choice((1, 1, rng.randint(2, 16), _log(rng, 17, 2048)))
    B = max(1, min(B, 10800 * 24 * 128 * 10 // (L * Hk * D)))
    while B * Hk * g * Nq * L > 24 * 2048 * 16896:
        if B > 1:
            B //= 2
        elif Nq > 1:
            Nq //= 2
        else:
            L //= 2
    return dict(op=op, B=B, Hq=Hk * g, Hk=Hk, D=D, page=page, L=L, Nq=min(Nq, L), causal=rng.random() < 0.7,
                ragged=rng.random() < 0.6)


def _lengths(n, B, ragged, least):
    """Lengths of a batch: all n, or spread from n / 2 to n."""
    if not ragged:
        return [n] * B
    return [max(least, n - (n // 2) * b // B) for b in range(B)]


def _need_exp(amax):
    """Least e in [-117, 119] with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)  # m in [0.5, 1): amax = 2m * 2^(x - 1); 448 = 1.75 * 2^8
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, SCALE_EXP_MIN)).clamp(SCALE_EXP_MIN, SCALE_EXP_MAX)


def _to_e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _value(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _filled(pages, H, page, D, g):
    """Codes and scales of pages that hold normal values, channels of unequal size."""
    x = torch.randn(pages, H, page, D, generator=g, device="cuda")
    x *= torch.exp(0.4 * torch.randn(1, H, 1, D, generator=g, device="cuda"))
    s = torch.exp2(_need_exp(x.abs().amax((2, 3))).float())
    return _to_e4m3(x / s[:, :, None, None]), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    B, D = case["B"], case["D"]
    if case["op"] == "rope":
        Hq, Hk, text = case["Hq"], case["Hk"], case["text"]
        grid = torch.cartesian_prod(*(torch.arange(n) for n in (case["t"], case["h"], case["w"])))
        N = text + grid.shape[0]
        pos = torch.zeros(B, N, 3, dtype=torch.int32)
        pos[:, text:] = grid.to(torch.int32)
        if grid.shape[0] == 1:  # a decode step: each sequence at a place of its own
            pos[:, text:] += torch.randint(0, 200000, (B, 1, 3), generator=torch.Generator().manual_seed(seed),
                                           dtype=torch.int32)
        s["pos"] = pos.cuda()
        s["dims"], s["theta"] = AXES[D], 10000.0
        dtype = DTYPES[case["dtype"]]
        if case["back"]:  # gradients as the attention leaves them, head-major
            s["q"] = torch.randn(B, Hq, N, D, generator=g, device="cuda").to(dtype)
            s["k"] = torch.randn(B, Hk, N, D, generator=g, device="cuda").to(dtype)
        else:  # slices of the token-major projection of q, k and v
            x = torch.randn(B, N, Hq + 2 * Hk, D, generator=g, device="cuda").to(dtype)
            s["q"], s["k"] = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
        return s
    H, page = case["Hk"], case["page"]
    if case["op"] == "cache":
        start = _lengths(case["start"], B, case["ragged"], 0)
        count = _lengths(case["N"], B, case["ragged"], 1)
        first = [a // page * page for a in start]
        end = [a + n for a, n in zip(start, count)]
        s["start"], s["count"], s["first"], s["end"] = (torch.tensor(v, dtype=torch.int32, device="cuda")
                                                        for v in (start, count, first, end))
        s["span"] = max(b - a for a, b in zip(first, end))
        x = torch.randn(B, case["N"], 3 * H, D, generator=g, device="cuda")
        x[:, ::97] *= 6.0  # tokens that raise a page's scale
        x = x.to(torch.bfloat16)
        s["k_new"] = x[:, :, H:2 * H].transpose(1, 2).contiguous()  # as rotary positions leave them
        s["v_new"] = x[:, :, 2 * H:].transpose(1, 2)                # a slice of the projection
        longest = max(end)
    else:
        lens = _lengths(case["L"], B, case["ragged"], case["Nq"])
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = torch.randn(B, case["Hq"], case["Nq"], D, generator=g, device="cuda").to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(D)
        longest = case["L"]
    per = -(-longest // page)
    pages = B * per + 3
    s["k8"], s["k_scale"] = _filled(pages, H, page, D, g)
    s["v8"], s["v_scale"] = _filled(pages, H, page, D, g)
    s["table"] = torch.randperm(pages, generator=g, device="cuda")[:B * per].view(B, per).to(torch.int32)
    return s


def _rope(x, pos, dims, theta, pairing, back):
    freq = torch.cat([theta ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d) for d in dims])
    axis = torch.cat([torch.full((d // 2,), a, device=x.device) for a, d in enumerate(dims)])
    angle = torch.remainder(pos.double()[:, None, :, axis] * freq, 2 * math.pi)
    cos, sin = angle.cos().float(), angle.sin().float()
    if back:
        sin = -sin
    D = x.shape[-1]
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if pairing == "adjacent" else (x[..., :D // 2], x[..., D // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.stack((a, b), -1).flatten(-2) if pairing == "adjacent" else torch.cat((a, b), -1)


def _write(s, new, codes, scales):
    """The pages that the new tokens touch, with old tokens rounded again where the scale grew."""
    B, H, N, D = new.shape
    page, start, end = s["page"], s["start"].long(), (s["start"] + s["count"]).long()
    slots = (start // page)[:, None] + torch.arange((N + page - 2) // page + 1, device=new.device)  # [B, T]
    touched = (slots * page < end[:, None]) & (slots < s["table"].shape[1])
    ids = s["table"].long().gather(1, slots.clamp(max=s["table"].shape[1] - 1))
    at = slots[:, :, None] * page + torch.arange(page, device=new.device)  # positions [B, T, page]
    fresh = (at >= start[:, None, None]) & (at < end[:, None, None])
    take = (at - start[:, None, None]).clamp(0, N - 1)
    x = new.float().transpose(1, 2)[torch.arange(B, device=new.device)[:, None, None], take]  # [B, T, page, H, D]
    x = torch.where(fresh[..., None, None], x, 0.0).transpose(2, 3)
    need = torch.exp2(_need_exp(x.abs().amax((3, 4))).float())
    old = scales[ids]
    has_old = (slots * page < start[:, None])[..., None]
    scale = torch.where(has_old, torch.maximum(old, need), need)
    kept = _value(codes[ids]) * (old / scale)[..., None, None]
    out = _to_e4m3(torch.where(fresh[:, :, None, :, None], x / scale[..., None, None], kept))
    codes.view(torch.uint8)[ids[touched]] = out.view(torch.uint8)[touched]
    scales[ids[touched]] = scale[touched]


def _read(s, codes, scales, first, end, n):
    """Tokens first .. first + n - 1 of each sequence, [B, H, n, D], zero from `end` on."""
    page = s["page"]
    at = first.long()[:, None] + torch.arange(n, device=codes.device)  # [B, n]
    slot = (at // page).clamp(max=s["table"].shape[1] - 1)
    ids = s["table"].long().gather(1, slot)
    x = _value(codes.view(torch.uint8)[ids, :, at % page]) * scales[ids][..., None]  # [B, n, H, D]
    return torch.where((at < end.long()[:, None])[..., None, None], x, 0.0).transpose(1, 2)


def run(s):
    if own:
        import unet_fa_fwd_gb300 as fa
    if s["op"] == "rope":
        if own:
            axes = fa.RopeAxes(s["dims"], s["theta"])
            if s["back"]:
                return fa.rope_bwd(s["q"], s["k"], s["pos"], axes, pairing=s["pairing"], token_major=True)
            return fa.rope(s["q"], s["k"], s["pos"], axes, pairing=s["pairing"])
        return tuple(_rope(x, s["pos"], s["dims"], s["theta"], s["pairing"], s["back"]).to(x.dtype)
                     for x in (s["q"], s["k"]))
    if own:
        cache = fa.KVCache8(s["k8"], s["v8"], s["k_scale"], s["v_scale"])
    if s["op"] == "cache":
        if own:
            fa.cache_write(cache, s["k_new"], s["v_new"], s["table"], s["start"], s["count"])
            return fa.cache_read(cache, s["table"], s["end"], s["span"], start=s["first"])
        got = []
        for new, codes, scales in (("k_new", "k8", "k_scale"), ("v_new", "v8", "v_scale")):
            _write(s, s[new], s[codes], s[scales])
            got.append(_read(s, s[codes], s[scales], s["first"], s["end"], s["span"]).to(torch.bfloat16))
        return tuple(got)
    if own:
        return fa.fwd_cache(s["q"], cache, s["table"], s["lens"], causal=s["causal"], scale=s["scale"])
    q = s["q"].float()
    B, Hq, Nq, D = q.shape
    Hk, L = s["Hk"], s["L"]
    lens = s["lens"].long()
    k, v = (_read(s, s[c], s[z], torch.zeros_like(lens), lens, L) for c, z in (("k8", "k_scale"), ("v8", "v_scale")))
    t = torch.matmul(q.view(B, Hk, Hq // Hk * Nq, D), k.transpose(2, 3)).view(B, Hk, Hq // Hk, Nq, L) * s["scale"]
    key = torch.arange(L, device=q.device)
    seen = key < lens[:, None, None]
    if s["causal"]:
        seen = seen & (key <= (lens[:, None] - Nq + torch.arange(Nq, device=q.device))[..., None])
    t = torch.where(seen[:, None, None], t, -math.inf)
    m = t.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(t - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hk, -1, L), v).view(B, Hk, Hq // Hk, Nq, D) / l.clamp(min=1e-30)
    lse = m + torch.log(l)
    return o.view(B, Hq, Nq, D).to(torch.bfloat16), lse.view(B, Hq, Nq)


def work(case):
    B, D = case["B"], case["D"]
    if case["op"] == "rope":
        n = B * (case["text"] + case["t"] * case["h"] * case["w"])
        width = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        values = n * (case["Hq"] + case["Hk"]) * D
        return dict(bytes=2 * width * values + 12 * n, flops=3 * values)
    H, page = case["Hk"], case["page"]
    if case["op"] == "cache":
        start = _lengths(case["start"], B, case["ragged"], 0)
        count = _lengths(case["N"], B, case["ragged"], 1)
        span = max(a % page + n for a, n in zip(start, count))
        held = sum(a % page + n for a, n in zip(start, count))  # tokens read back
        scales = sum(-(-(a % page + n) // page) for a, n in zip(start, count))
        values = 2 * H * D * (3 * sum(count) + held + 2 * B * span)
        return dict(bytes=values + 3 * 2 * H * 4 * scales, flops=2 * H * D * 3 * sum(count))
    lens = _lengths(case["L"], B, case["ragged"], case["Nq"])
    Nq, Hq = case["Nq"], case["Hq"]
    pairs = sum(Nq * n - (Nq * (Nq - 1) // 2 if case["causal"] else 0) for n in lens)
    scales = sum(-(-n // page) for n in lens)
    return dict(bytes=2 * H * D * sum(lens) + 2 * H * 4 * scales + B * Hq * Nq * (4 * D + 4),
                flops=4 * D * Hq * pairs)


def _ladder():
    """Every value of e4m3 from its definition: sign, four exponent bits (bias 7), three of mantissa."""
    v = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _nearest(x):
    """x (64 bits) to the nearest e4m3 value, ties to the even code, saturating."""
    ladder = _ladder()
    a = x.abs().contiguous()
    hi = torch.searchsorted(ladder, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = ladder[hi] - a, a - ladder[lo]
    i = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    i = torch.where(a >= ladder[126], torch.full_like(i, 126), i)
    return torch.sign(x) * ladder[i]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        phase = []
        for a, d in enumerate(s["dims"]):
            for j in range(d // 2):
                phase.append(s["pos"][:, :, a].double() * s["theta"] ** (-2.0 * j / d))
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.stack(phase, -1))
        turn = (turn.conj() if case["back"] else turn)[:, None]
        got = []
        for x in (s["q"], s["k"]):
            out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            half = case["D"] // 2
            for h in range(x.shape[1]):
                y = x[:, h:h + 1].double()
                if case["pairing"] == "adjacent":
                    z = torch.view_as_complex(y.reshape(*y.shape[:3], half, 2).contiguous()) * turn
                    out[:, h:h + 1] = torch.view_as_real(z).flatten(-2)
                else:
                    z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * turn
                    out[:, h:h + 1, :, :half], out[:, h:h + 1, :, half:] = z.real, z.imag
            got.append(out)
        return got
    B, H, page, D = case["B"], case["Hk"], case["page"], case["D"]
    table = s["table"].tolist()
    if case["op"] == "cache":
        got = []
        start, count, first, end = (s[n].tolist() for n in ("start", "count", "first", "end"))
        for new, codes, scales in ((s["k_new"], s["k8"], s["k_scale"]), (s["v_new"], s["v8"], s["v_scale"])):
            out = torch.zeros(B, H, s["span"], D, dtype=torch.float64, device="cuda")
            for b in range(B):
                at = first[b]
                while at < end[b]:
                    old = max(0, min(start[b] - at, page))  # tokens that the page held before
                    lo, hi = at + old - start[b], min(at + page, end[b]) - start[b]
                    x = new[b, :, lo:hi].double()
                    # least power of two s with max |x| <= 448 s
                    most = x.abs().amax((1, 2)).clamp(min=448.0 * 2.0 ** SCALE_EXP_MIN)
                    z = torch.exp2(torch.ceil(torch.log2(most / 448.0)))
                    z = torch.where(most > 448.0 * z, 2 * z, torch.where(most <= 224.0 * z, z / 2, z))
                    id_ = table[b][at // page]
                    if old:
                        was = scales[id_].double()
                        z = torch.maximum(z, was)
                        kept = codes[id_, :, :old].double() * was[:, None, None]
                        out[b, :, at - first[b]:at - first[b] + old] = (_nearest(kept / z[:, None, None])
                                                                         * z[:, None, None])
                    out[b, :, at + old - first[b]:at - first[b] + old + hi - lo] = (_nearest(x / z[:, None, None])
                                                                                     * z[:, None, None])
                    at += page
            got.append(out)
        return got
    Hq, Nq, L = case["Hq"], case["Nq"], case["L"]
    if 2 * Hq * Nq * sum(s["lens"].tolist()) * D > 2e12:
        return None
    o = torch.zeros(B, Hq, Nq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Hq, Nq, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        ids = torch.tensor(table[b][:-(-n // page)], device="cuda")
        k, v = ((c.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * z[ids].double()[:, :, None, None])
                .transpose(0, 1).reshape(H, -1, D)[:, :n] for c, z in ((s["k8"], s["k_scale"]), (s["v8"], s["v_scale"])))
        for h in range(Hq):
            t = s["q"][b, h].double() @ k[h * H // Hq].T * s["scale"]
            if case["causal"]:
                t = t + torch.full((Nq, n), -math.inf, dtype=torch.float64, device="cuda").triu(n - Nq + 1)
            lse[b, h] = torch.logsumexp(t, -1)
            o[b, h] = torch.exp(t - lse[b, h][:, None]) @ v[h * H // Hq]
    return [o, lse]
