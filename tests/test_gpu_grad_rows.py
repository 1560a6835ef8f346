"""Gradients of rows that masks leave in an unusual state: wholly under a large finite
mask, or without a key while they hold numbers that are not finite.

A row's softmax does not change when a constant is taken off its scores, so the 64-bit
definition takes each row's largest mask value off first; O and LSE are rounded from it
as the forward's are.
"""
import math
import os
import subprocess
import sys

import pytest
import torch

import unet_fa_fwd_gb300 as fa

from . import grad_ref as ref
from .test_gpu_bwd import _full_mask, _inputs, _rand

pytestmark = pytest.mark.gpu

INF = math.inf
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0


# ---- rows wholly under a large finite mask ----

def _check_shifted(B, Hq, Hk, Nq, Nk, D, causal, seed=1, **mask):
    """Tolerances as in the tests of ordinary masks, and 2^-9 of P (in its terms, and in the norm) for rows of
    |LSE| below 2^14: LSE is within 2^-11 (half its step), L = LSE log2(e) and mask log2(e) within 2^-10 each in
    the log2 domain, so P within 2^-11 + 2 ln(2) 2^-10 < 2^-9 of itself.  Rows past that are summed again from
    scores whole, whose errors are those of ordinary rows."""
    m = mask["key_mask"][:, None, None].expand(B, 1, Nq, Nk) if "key_mask" in mask else mask["full_mask"]
    seen = m > -INF
    if causal:
        seen = seen & torch.ones(Nq, Nk, dtype=torch.bool, device="cuda").tril()
    top = m.double().masked_fill(~seen, -INF).amax(-1, keepdim=True)
    shift = torch.where(top.isfinite(), top, 0.0)
    even = (m.double() - shift).masked_fill(~seen, -INF)
    q, k, v, do = (_rand((B, H, N, D), seed + i) for i, (H, N) in enumerate(((Hq, Nq), (Hk, Nk), (Hk, Nk), (Hq, Nq))))
    scale = 1 / math.sqrt(D)
    o, lse = ref.attend(q, k, v, scale, full_mask=even)
    x = dict(dout=do, q=q, k=k, v=v, out=o.to(torch.bfloat16), scale=scale)
    low = (lse + shift[..., 0]).float()
    again = ((low.abs() >= 2 ** 14) & low.isfinite())[..., None]  # (O is not used: delta is the definition's)
    got = fa.bwd(**dict(x, out=x["out"].masked_fill(again, math.nan)), lse=low, causal=causal, **mask)
    x["out"] = torch.where(again, o, x["out"].double())
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0
    want, size, fine = ref.attend_bwd(**x, lse=lse, full_mask=even)
    for name, y, w, s, f in zip(("dq", "dk", "dv"), got, want, size, fine):
        err = (y.double() - w).abs()
        tol = 2.0 ** -8 * w.abs() + (2.0 ** -8 + 2.0 ** -13 + 2.0 ** -9) * s + 2.0 ** -16 * f
        assert bool((err <= tol).all()), (name, float((err - tol).max()), float(err.max()))
        assert float(err.norm()) <= (5e-3 + 2.0 ** -9) * float(w.norm()), (name, float(err.norm() / w.norm()))


LARGE = [-1e4, -65504.0, -1e6, -1e9, -1e30, -2e38, 1e9]  # (past 2.3e38 they leave fp32's range in the log2 domain)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("c", LARGE)
@pytest.mark.parametrize("size", [(2, 2, 2, 130, 77), (3, 4, 2, 300, 400), (2, 1, 1, 1, 33)])
def test_entries_wholly_under_a_large_key_mask(D, c, size):
    B, Nk = size[0], size[4]
    m = torch.zeros(B, Nk, device="cuda")
    m[0, Nk // 2:] = -abs(c)            # ordinary padding
    m[1] = c                            # a whole entry
    m[1, Nk // 3] = -INF
    if B > 2:
        m[2, 5:] = c                    # five ordinary keys, or all but five above the others
    _check_shifted(*size, D, False, key_mask=m)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("c", LARGE[1:5])
@pytest.mark.parametrize("size,pad", [((2, 2, 2, 260, 260), 100), ((1, 4, 1, 700, 700), 300), ((1, 1, 1, 2100, 2100), 140)])
def test_padding_ahead_of_a_causal_sequence(D, c, size, pad):
    """The first rows see padding only; those behind see both."""
    m = torch.zeros(size[0], size[4], device="cuda")
    m[0, :pad] = c
    _check_shifted(*size, D, True, key_mask=m)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("c", LARGE)
@pytest.mark.parametrize("size,heads,causal", [((2, 2, 2, 130, 77), 1, False), ((1, 4, 2, 257, 400), 4, True),
                                               ((2, 2, 1, 3, 33), 2, False), ((1, 1, 1, 1500, 1100), 1, False)])
def test_rows_wholly_under_a_large_additive_mask(D, c, size, heads, causal):
    B, Hq, Hk, Nq, Nk = size
    m = _full_mask("add", B, heads, Nq, Nk, 4)
    m[:, :, Nq // 2:Nq // 2 + 20] = c   # whole rows, and one of two heights
    m[:, :, -1] = c
    m[:, :, -1, Nk // 2:] = -abs(c) * 1.1
    m[..., 0, :, 3] = -INF
    m[0, 0, :, Nk // 4] = -abs(c)       # a column that ordinary rows do not see
    _check_shifted(*size, D, causal, full_mask=m)


@pytest.mark.parametrize("c", [-1e4, -1e6, -1e9, -1e30])
@pytest.mark.parametrize("kind", ["key", "add"])
def test_with_the_forwards_own_results(c, kind):
    """Rows wholly at one value: the gradients are those of no mask, although the forward's O is of scores that the
    mask's step has rounded.  Both are within P's 2^-9 (the rows at -1e4), its rounding and the results'."""
    B, H, N, D = 2, 2, 300, 64
    q, k, v, do = (_rand((B, H, N, D), i) for i in range(4))
    mask = dict(key_mask=torch.full((B, N), c, device="cuda")) if kind == "key" else dict(
        full_mask=torch.full((B, 1, N, N), c, device="cuda"))
    out, lse = fa.fwd_ex(q, k, v, **mask)
    got = fa.bwd(do, q, k, v, out, lse, **mask)
    o, lse = ref.attend(q, k, v, 1 / math.sqrt(D))
    want = ref.attend_bwd(do, q, k, v, o, lse, 1 / math.sqrt(D))[0]
    for a, b in zip(got, want):
        assert float((a.double() - b).norm()) <= (5e-3 + 2.0 ** -9) * float(b.norm())


@pytest.mark.parametrize("D", [32, 128])
def test_rows_that_their_scores_make_large(D):
    """|LSE| past 2^14 from scores, under masks that add nothing: bit for bit what no mask gives."""
    B, H, N = 1, 2, 200
    x = _inputs(B, H, H, N, N, D, scale=4000.0)
    assert float(x["lse"].abs().median()) > 2 ** 14
    want = fa.bwd(**x)
    assert all(bool(y.isfinite().all()) for y in want)
    for mask in (dict(key_mask=torch.zeros(B, N, device="cuda")), dict(full_mask=torch.zeros(B, 1, N, N, device="cuda"))):
        assert all(torch.equal(a, b) for a, b in zip(fa.bwd(**x, **mask), want))


def test_large_masks_repeat_and_agree_with_none():
    """All rows at one large value: the gradients of no mask, but for the rows' own normaliser; twice the same."""
    B, H, N, D = 1, 3, 500, 64
    x = _inputs(B, H, H, N, N, D)
    x["lse"] = x["lse"] - 1e9
    m = torch.full((B, 1, N, N), -1e9, device="cuda")
    one, two = fa.bwd(**x, full_mask=m), fa.bwd(**x, key_mask=m[:, 0, 0].contiguous())
    plain = fa.bwd(**dict(x, lse=x["lse"] * 0 + _inputs(B, H, H, N, N, D)["lse"]))
    again = fa.bwd(**x, full_mask=m)
    assert all(torch.equal(a, b) for a, b in zip(one, again))
    for a, b, c in zip(one, two, plain):
        # P within 2^-13 of itself either way; both results, P and dS rounded to bf16 alike or one step apart
        for y in (a, b):
            assert float((y.double() - c.double()).norm()) <= 5e-3 * float(c.double().norm())


# ---- rows without a key ----

def _bad_rows(x, rows, value):
    """What padding rows hold: anything, in all of their tensors."""
    y = dict(x)
    for n in ("q", "dout", "out"):
        y[n] = x[n].clone()
        y[n][:, :, rows] = value
        y[n][:, :, rows, ::3] = -value
    if x.get("dlse") is not None:
        y["dlse"] = x["dlse"].clone()
        y["dlse"][:, :, rows] = value
    return y


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bool", "u8", "add", "lowest"])
@pytest.mark.parametrize("size,heads,causal", [((2, 2, 2, 130, 77), 1, False), ((1, 4, 2, 400, 257), 4, True),
                                               ((1, 2, 1, 900, 700), 1, False), ((2, 1, 1, 3, 200), 1, False)])
@pytest.mark.parametrize("value", [math.nan, INF, 3e38])
def test_rows_without_a_key_may_hold_anything(D, kind, size, heads, causal, value):
    B, Hq, Hk, Nq, Nk = size
    m = _full_mask(kind, B, heads, Nq, Nk, 4)
    rows = sorted({Nq // 3, *range(Nq // 2, Nq // 2 + Nq // 10), Nq - 1})
    m[:, :, rows] = {"add": -INF, "lowest": torch.finfo(torch.float32).min}.get(kind, 0)
    plain = m.masked_fill(m < -1e38, -INF) if kind == "lowest" else m
    x = dict(_inputs(*size, D, full_mask=plain, causal=causal, dlse=True), full_mask=m)
    assert bool((x["lse"][:, :, rows] == -INF).all())
    want = fa.bwd(**x)
    got = fa.bwd(**_bad_rows(x, rows, value))
    assert all(bool(y.isfinite().all()) for y in want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((got[0][:, :, rows] == 0).all())


@pytest.mark.parametrize("D", [64, 128])
def test_an_entry_without_a_key_may_hold_anything(D):
    """A whole entry of a padded batch; ordinary keys of the other one are padding too."""
    B, H, Nq, Nk = 2, 2, 300, 500
    for low in (-INF, torch.finfo(torch.float32).min):
        m = torch.zeros(B, Nk, device="cuda")
        m[0, 200:], m[1] = -INF, -INF
        x = _inputs(B, H, H, Nq, Nk, D, key_mask=m, dlse=True)
        x["key_mask"] = m.masked_fill(m == -INF, low)
        want = fa.bwd(**x)
        bad = _bad_rows(x, list(range(Nq)), math.nan)
        for n in ("q", "dout", "out", "dlse"):
            bad[n][0] = x[n][0]
        assert all(torch.equal(a, b) for a, b in zip(fa.bwd(**bad), want))


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("kind", ["add", "key", "bool"])
def test_strided_tensors_streams_and_graphs(D, kind):
    """Both kinds of row in tensors of other strides, on another stream and captured: bit for bit the same."""
    B, Hq, Hk, N = 2, 4, 2, 330
    if kind == "key":
        masks = dict(key_mask=torch.zeros(B, N, device="cuda"), causal=True)
        masks["key_mask"][0, :40], masks["key_mask"][1, :140] = -INF, -1e9
        odd = list(range(40))
    else:
        m = _full_mask(kind, B, 1, N, N, 4)
        if kind == "add":
            m[:, :, 200:230] = -1e9
        m[:, :, 280:300] = -INF if kind == "add" else False
        masks, odd = dict(full_mask=m), list(range(280, 300))
    x = _inputs(B, Hq, Hk, N, N, D, **masks, dlse=True)
    x["dlse"] = torch.where(x["lse"] == -INF, math.nan, x["dlse"])
    for n in ("q", "dout", "out"):
        x[n][0, :, odd] = math.nan
    want = fa.bwd(**x)
    assert all(bool(y.isfinite().all()) for y in want)
    y = dict(x)
    for n in ("dout", "q", "k", "v", "out"):  # token-major, every other head of wider rows
        b, h, t, d = x[n].shape
        wide = torch.full((b, t, 2 * h, d + 8), math.nan, dtype=torch.bfloat16, device="cuda")
        y[n] = wide[:, :, ::2, 8:].transpose(1, 2)
        y[n].copy_(x[n])
    assert all(torch.equal(a, b) for a, b in zip(fa.bwd(**y, token_major=True), want))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fa.bwd(**y, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.bwd(**y)
    for g in got:
        g.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


CHILD = r'''
import sys, torch
sys.path.insert(0, ROOT)
import unet_fa_fwd_gb300 as fa
from tests.test_gpu_grad_rows import _check_shifted, test_rows_without_a_key_may_hold_anything
assert fa.debug_build(), "the debug library was not loaded"
torch.cuda.set_device(0)
for D in (32, 64, 128):
    m = torch.zeros(2, 300, device="cuda")
    m[0, 200:], m[1] = -1e9, -1e6
    _check_shifted(2, 4, 2, 260, 300, D, False, key_mask=m)
    test_rows_without_a_key_may_hold_anything(D, "add", (1, 4, 2, 400, 257), 4, True, float("nan"))
    torch.cuda.synchronize()
    st, rec = fa.read_device_status(), fa.debug_report()
    assert st == 0 and rec == [0] * 8, (D, st, rec)
print("debug build: no violation")
'''


def test_debug_build_reports_no_violation():
    r = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT))], cwd=ROOT,
                       env=dict(os.environ, FA_DEBUG="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "no violation" in r.stdout
