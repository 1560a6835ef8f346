"""The attention's gradient on the GPU against its 64-bit definition, from the same
O and LSE (computed in 64 bits and rounded as the forward's are).

Tolerances.  P and dS are rounded to bf16 for the products that take them: half a
step, 2^-8, of each term.  Scores are fp32 sums of at most 128 exact products of
size below 2^5 (log2 domain), so t is within 2^-15, which moves P by less than 2^-15
of itself; dP - delta is within 129 additions' 2^-24 of the sizes of its terms, 2^-17.
So |error| <= 2^-8 |x| (the result's own rounding) + (2^-8 + 2^-13) sum |terms|
+ 2^-16 sum P (sizes of the terms of dP and delta) |other factor|.
That bound has every rounding at its worst at once.  Over a whole result of random
inputs the roundings are independent: each is at most 2^-8 / sqrt(3) = 2.3e-3 of a
term in the mean square, the result's own and its terms' together 3.2e-3 of the
result's norm, which a lost key or query of a few hundred passes by far: the norm of
the error is held to 5e-3.
"""
import math

import pytest
import torch

import unet_fa_fwd_gb300 as fa

from . import grad_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0


def _rand(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _inputs(B, Hq, Hk, Nq, Nk, D, seed=1, scale=None, dlse=False, **masks):
    q, k, v, do = (_rand((B, H, N, D), seed + i) for i, (H, N) in enumerate(((Hq, Nq), (Hk, Nk), (Hk, Nk), (Hq, Nq))))
    scale = 1 / math.sqrt(D) if scale is None else scale
    o, lse = ref.attend(q, k, v, scale, **masks)
    return dict(dout=do, q=q, k=k, v=v, out=o.to(torch.bfloat16), lse=lse.float(), scale=scale,
                dlse=_rand((B, Hq, Nq), seed + 9, torch.float32) if dlse else None, **masks)


def _check(got, x, norm=True):
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0
    want, size, fine = ref.attend_bwd(**x)
    for name, y, w, s, f in zip(("dq", "dk", "dv"), got, want, size, fine):
        assert y.dtype == torch.bfloat16 and y.shape == w.shape
        err = (y.double() - w).abs()
        tol = 2.0 ** -8 * w.abs() + (2.0 ** -8 + 2.0 ** -13) * s + 2.0 ** -16 * f
        assert bool((err <= tol).all()), (name, float((err - tol).max()), float(err.max()))
        if norm and float(w.norm()) > 1e-3 * float(f.norm()):
            assert float(err.norm()) <= 5e-3 * float(w.norm()), (name, float(err.norm() / w.norm()))


def _bwd(x, **kw):
    return fa.bwd(**x, **kw)


SIZES = [(1, 1, 1, 1, 1), (2, 3, 3, 128, 128), (1, 2, 2, 127, 129), (2, 3, 1, 77, 130), (1, 8, 2, 257, 300),
         (1, 2, 2, 1, 500), (1, 1, 1, 700, 1), (3, 4, 4, 384, 64), (1, 1, 1, 2000, 300), (1, 1, 1, 130, 2500)]


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("causal", [False, True])
def test_against_definition(D, size, causal):
    x = _inputs(*size, D, causal=causal, dlse=size[3] == 1 or size[4] == 1)
    _check(_bwd(x), x)


def _key_mask(B, Nk, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = 0.5 * torch.randn(B, Nk, generator=g, device="cuda")
    m[torch.rand(B, Nk, generator=g, device="cuda") < 0.2] = -math.inf
    m[0, Nk // 2:] = -math.inf
    return m


def _full_mask(kind, B, heads, Nq, Nk, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    keep = torch.rand(B, heads, Nq, Nk, generator=g, device="cuda") < 0.7
    keep[:, :, Nq // 3] = False           # a row that sees nothing
    keep[:, :, :, Nk // 2] = False        # a key that nobody sees
    if kind == "bool":
        return keep
    if kind == "u8":
        return keep.to(torch.uint8) * 3
    m = torch.randn(B, heads, Nq, Nk, generator=g, device="cuda")
    return m.masked_fill(~keep, -math.inf if kind == "add" else torch.finfo(torch.float32).min)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("size", [(2, 2, 2, 130, 77), (1, 4, 2, 257, 400), (2, 1, 1, 1, 33), (1, 2, 2, 900, 129)])
@pytest.mark.parametrize("causal", [False, True])
def test_key_mask(D, size, causal):
    B, Nk = size[0], size[4]
    x = _inputs(*size, D, key_mask=_key_mask(B, Nk, 3), causal=causal, dlse=True)
    _check(_bwd(x), x)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bool", "u8", "add", "lowest"])
@pytest.mark.parametrize("size,shared", [((2, 2, 2, 130, 77), True), ((1, 4, 2, 257, 400), False),
                                         ((2, 2, 1, 3, 33), False), ((1, 2, 2, 900, 128), True)])
@pytest.mark.parametrize("causal", [False, True])
def test_full_mask(D, kind, size, shared, causal):
    B, Hq, Hk, Nq, Nk = size
    m = _full_mask(kind, B, 1 if shared else Hq, Nq, Nk, 4)
    if kind == "lowest":  # as -inf: past fp32's range in the log2 domain, as in the forward
        x = _inputs(*size, D, full_mask=m.masked_fill(m < -1e38, -math.inf), causal=causal, dlse=True)
        got = _bwd(dict(x, full_mask=m))
    else:
        x = _inputs(*size, D, full_mask=m, causal=causal, dlse=True)
        got = _bwd(x)
    _check(got, x)


def test_rows_and_keys_that_meet_nothing():
    """Rows without a key and keys without a row have gradients of exactly 0, in cut units too."""
    B, H, Nq, Nk, D = 1, 1, 1500, 700, 64
    keep = torch.ones(B, 1, Nq, Nk, dtype=torch.bool, device="cuda")
    keep[:, :, 200:460] = False
    keep[..., 100:300] = False
    x = _inputs(B, H, H, Nq, Nk, D, full_mask=keep)
    dq, dk, dv = _bwd(x)
    _check((dq, dk, dv), x)
    assert bool((dq[:, :, 200:460] == 0).all())
    assert bool((dk[:, :, 100:300] == 0).all()) and bool((dv[:, :, 100:300] == 0).all())
    x = _inputs(B, H, H, 200, 900, D, causal=True)  # keys past the last query
    dq, dk, dv = _bwd(x)
    _check((dq, dk, dv), x)
    assert bool((dk[:, :, 200:] == 0).all()) and bool((dv[:, :, 200:] == 0).all())
    x = _inputs(B, H, H, 300, 300, D, full_mask=torch.zeros(B, 1, 300, 300, dtype=torch.bool, device="cuda"))
    assert bool((x["lse"] == -math.inf).all())
    assert all(bool((y == 0).all()) for y in _bwd(x))


@pytest.mark.parametrize("scale", [0.0, -0.3, 0.02, 2.0])
def test_scales(scale):
    x = _inputs(1, 2, 2, 200, 333, 64, scale=scale)
    _check(_bwd(x), x, norm=scale != 0)


def test_large_scores():
    """Scores of several thousand either way: nearly one-hot rows, and tails past Nk where exp(-LSE) overflows.

    What t - L is off by, in the log2 domain, with T = scale log2(e) sum |q k| (up to 2^13 here): S is a sum of
    64 exact products in four steps, each within 2^-23 of the sizes added so far however it aligns them, so 2^-20
    T holds it; scale log2(e) is rounded (2^-24 T), L is rounded from LSE log2(e) (2^-23 |L| with the constant's
    rounding), t - L once more (2^-24 of itself, at most 2^-24 (T + |L|)).  P moves by 2^that - 1 of itself.  (2^-12
    of P, as this test assumed first, holds for scores of up to 2^7 only.)  P below 2^-126, fp32's least normal
    number, is 0, and dS likewise: 2^-125 of P, times (1 + |dP - delta|) in dS, holds both."""
    x = _inputs(1, 2, 2, 150, 190, 64, scale=16.0)
    x["k"] = x["k"] - 4 * x["q"][:, :, :1].sign()  # the first row's scores are all far below zero
    x["out"], x["lse"] = ref.attend(x["q"], x["k"], x["v"], 16.0)
    x["out"], x["lse"] = x["out"].to(torch.bfloat16), x["lse"].float()
    got = _bwd(x)
    torch.cuda.synchronize()
    want, size, fine = ref.attend_bwd(**x)
    T = lambda y: y.transpose(2, 3)  # noqa: E731
    q, k, v, do = (x[n].double() for n in ("q", "k", "v", "dout"))
    lse = x["lse"].double()[..., None]
    log2e = math.log2(math.e)
    terms = (q.abs() @ T(k.abs())) * 16.0 * log2e
    off = 2.0 ** -20 * terms + 2.0 ** -24 * terms + 2.0 ** -23 * lse.abs() * log2e + 2.0 ** -24 * (
        terms + lse.abs() * log2e)
    p = torch.exp(ref.scores(x["q"], x["k"], 16.0) - lse)
    dp = p * (torch.exp2(off) - 1) + 2.0 ** -125
    ds = dp * (do @ T(v) - (do * x["out"].double()).sum(-1, keepdim=True)).abs() + 2.0 ** -125
    moved = (ds @ k.abs() * 16, T(ds) @ q.abs() * 16, T(dp) @ do.abs())
    for y, w, s, f, m in zip(got, want, size, fine, moved):
        assert bool(y.isfinite().all())
        err = (y.double() - w).abs()
        assert bool((err <= 2.0 ** -8 * w.abs() + (1 + 2.0 ** -8) * (2.0 ** -8 * s + m + 2.0 ** -16 * f)).all())


@pytest.mark.parametrize("D", [32, 64, 128])
def test_cut_and_whole_units_many_heads(D):
    """More units than SMs, the last ones cut; shared key heads."""
    x = _inputs(2, 16, 4, 1100, 1300, D)
    _check(_bwd(x), x)
    x = _inputs(2, 16, 4, 1300, 1300, D, causal=True)
    _check(_bwd(x), x)


def test_repeats_bit_for_bit():
    x = _inputs(1, 6, 3, 1500, 1111, 128, causal=True)
    one = _bwd(x)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(one, _bwd(x)))


def _strided(shape, seed, kind):
    """A [B, H, N, D] tensor laid out another way."""
    B, H, N, D = shape
    if kind == "token":
        return _rand((B, N, H, D), seed).transpose(1, 2)
    if kind == "packed":  # every other head of a buffer with rows of D + 8
        return _rand((B, N, 2 * H, D + 8), seed)[:, :, ::2, 8:].transpose(1, 2)
    return _rand((H, B, N, D), seed).transpose(0, 1)  # head-major over the batch


@pytest.mark.parametrize("kind", ["token", "packed", "heads"])
@pytest.mark.parametrize("D", [32, 128])
def test_strided_inputs_and_outputs(kind, D):
    B, Hq, Hk, Nq, Nk = 2, 4, 2, 150, 270
    x = _inputs(B, Hq, Hk, Nq, Nk, D)
    for i, name in enumerate(("dout", "q", "k", "v", "out")):
        t = _strided(x[name].shape, 20 + i, kind)
        t.copy_(x[name])
        x[name] = t
    want = _bwd({n: t.contiguous() if n in ("dout", "q", "k", "v", "out") else t for n, t in x.items()})
    got = _bwd(x, token_major=kind == "token")
    _check(got, x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(fa.bwd_workspace_bytes(B, Hq, Hk, Nq, Nk, D), dtype=torch.uint8, device="cuda")
    wide = torch.full((B, Nq + 2, Hq, D + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    dq = wide[:, 1:-1, :, 8:D + 8].transpose(1, 2)
    both = torch.full((2, B, Hk, Nk + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    dk, dv = both[0, :, :, :Nk], both[1, :, :, :Nk]
    args = {n: x[n] for n in ("key_mask", "full_mask", "causal", "scale", "dlse") if n in x}
    fa.fa_bwd(*(x[n] for n in ("dout", "q", "k", "v", "out", "lse")), dq, dk, dv, ws, **args)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), want))
    assert bool((wide[:, 0] == 7).all()) and bool((wide[:, -1] == 7).all())
    assert bool((wide[..., :8] == 7).all()) and bool((wide[..., D + 8:] == 7).all()) and bool((both[:, :, :, Nk] == 7).all())


def test_refusals_on_the_gpu():
    x = _inputs(1, 2, 2, 40, 40, 64)
    with pytest.raises(RuntimeError, match="INVALID"):   # rows off 16 bytes
        _bwd(dict(x, q=_rand((1, 2, 40, 65), 3)[..., 1:]))
    with pytest.raises(RuntimeError, match="INVALID"):   # a broadcast axis
        _bwd(dict(x, dout=_rand((1, 1, 40, 64), 3).expand(1, 2, 40, 64)))
    with pytest.raises(ValueError, match="last axis"):
        _bwd(dict(x, dout=torch.ones((), dtype=torch.bfloat16, device="cuda").expand(1, 2, 40, 64)))
    with pytest.raises(ValueError, match="shape"):
        _bwd(dict(x, lse=x["lse"][:, :1].contiguous()))
    with pytest.raises(RuntimeError, match="INVALID"):   # 3 query heads on 2 key heads
        _bwd(dict(_inputs(1, 3, 3, 40, 40, 64), k=x["k"], v=x["v"]))


def test_gradient_is_that_of_differences():
    """Directional differences of the 64-bit forward; the loss weighs O and LSE."""
    B, Hq, Hk, Nq, Nk, D = 1, 4, 2, 60, 90, 64
    x = _inputs(B, Hq, Hk, Nq, Nk, D, dlse=True, causal=True)
    x["out"] = ref.attend(x["q"], x["k"], x["v"], x["scale"], causal=True)[0].to(torch.bfloat16)
    got = _bwd(x)
    step = 2.0 ** -12
    for seed in range(3):
        d = [_rand(x[n].shape, 50 + seed, torch.float64) for n in "qkv"]

        def loss(sign):
            o, lse = ref.attend(*(x[n].double() + sign * step * y for n, y in zip("qkv", d)), x["scale"], causal=True)
            return (o * x["dout"].double()).sum() + (lse * x["dlse"].double()).sum()

        moved = (loss(1) - loss(-1)) / (2 * step)
        along = sum((a.double() * b).sum() for a, b in zip(got, d))
        # roundings of 2^-8 of the terms, independent: a few times 2^-8 of the root of the sum of squares; O's own
        # rounding moves delta by 2^-8 |O . dO|
        size = math.sqrt(sum(float((a.double() * b).square().sum()) for a, b in zip(got, d)))
        assert abs(float(moved - along)) <= 8 * 2.0 ** -8 * size


def test_other_stream_graph_and_two_at_once():
    x, y = _inputs(1, 4, 2, 700, 500, 128, seed=1), _inputs(1, 4, 2, 700, 500, 128, seed=30)
    want, want_y = _bwd(x), _bwd(y)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got, got_y = _bwd(x, stream=a), _bwd(y, stream=b)
    a.synchronize(), b.synchronize()
    assert all(torch.equal(u, w) for u, w in zip(got + got_y, want + want_y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _bwd(x)
    for n in ("dout", "q", "k", "v", "out", "lse"):
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, w) for u, w in zip(got, want_y))


def test_withheld_tile_times_out_and_context_survives(monkeypatch):
    x = _inputs(1, 4, 4, 900, 900, 128)
    want = _bwd(x)
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0
    monkeypatch.setenv("FA_FAULT_INJECT", "stall")
    monkeypatch.setenv("FA_WAIT_TIMEOUT_MS", "100")
    _bwd(x)
    torch.cuda.synchronize()
    assert fa.read_device_status() == fa.binding.FA_ERR_TIMEOUT
    monkeypatch.delenv("FA_FAULT_INJECT")
    monkeypatch.delenv("FA_WAIT_TIMEOUT_MS")
    assert all(torch.equal(a, b) for a, b in zip(_bwd(x), want))
