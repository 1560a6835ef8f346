"""An attention layer's training step, its operators together as they are used: norm
of queries and keys with the rotary positions, attention, and the gradients of both;
masks that start at any byte; the debug build's checks of the gradient's kernels.

Each stage is held to its 64-bit definition on what the stage before it left (the
tolerances of those operators' own tests), and the whole to differences of the
64-bit layer.
"""
import math
import os
import subprocess
import sys

import pytest
import torch

import unet_fa_fwd_gb300 as fa

from . import grad_ref as ref
from .test_gpu_bwd import _check as _check_bwd
from .test_gpu_bwd import _inputs
from .test_gpu_norm_rope import DIMS, EPS, _check_backward, _check_forward

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def _layer(B, Hq, N, D, seed=1):
    """Slices of a token-major projection, as a model holds them."""
    x = _rand((B, N, 3 * Hq, D), seed)
    q, k, v = (x[:, :, i * Hq:(i + 1) * Hq].transpose(1, 2) for i in range(3))
    w = [1 + 0.3 * _rand((D,), seed + i, torch.float32) for i in (1, 2)]
    pos = torch.stack(torch.meshgrid(*(torch.arange(n, dtype=torch.int32, device="cuda") for n in (1, 1, N)),
                                     indexing="ij"), -1).view(N, 3).contiguous()
    return q, k, v, w[0], w[1], pos, _rand((B, N, Hq, D), seed + 3).transpose(1, 2)


def _step(q0, k0, v, wq, wk, pos, dout, axes, **masks):
    """The calls of a training step; everything they leave."""
    q, k = fa.norm_rope(q0, k0, pos, axes, wq, wk, eps=EPS)
    vc = v.contiguous()
    out, lse = fa.fwd_ex(q, k, vc, **masks)
    dq, dk, dv = fa.bwd(dout, q, k, v, out, lse, token_major=True, **masks)
    return (q, k, out, lse, dq, dk, dv) + fa.norm_rope_bwd(dq, dk, q0, k0, pos, axes, wq, wk, eps=EPS,
                                                           token_major=True)


@pytest.mark.parametrize("D,N,masks", [(32, 77, {}), (64, 300, dict(causal=True)), (128, 200, {}),
                                       (128, 131, "bool")])
def test_a_training_step(D, N, masks):
    B, H = 2, 3
    axes = fa.RopeAxes(DIMS[D])
    q0, k0, v, wq, wk, pos, dout = _layer(B, H, N, D)
    if masks == "bool":
        keep = torch.rand(B, 1, N, N, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda") < 0.6
        keep[:, :, N // 2] = False
        masks = dict(full_mask=keep)
    q, k, out, lse, dq, dk, dv, dq0, dk0, dwq, dwk = _step(q0, k0, v, wq, wk, pos, dout, axes, **masks)
    _check_forward(q, q0, wq, pos, D, "adjacent")
    _check_forward(k, k0, wk, pos, D, "adjacent")
    _check_bwd((dq, dk, dv), dict(dout=dout, q=q, k=k, v=v, out=out, lse=lse, scale=1 / math.sqrt(D), **masks))
    _check_backward(dq0, dwq, dq, q0, wq, pos, D, "adjacent")
    _check_backward(dk0, dwk, dk, k0, wk, pos, D, "adjacent")


def test_the_step_is_the_gradient_of_the_layer():
    """Differences of the whole layer in 64 bits along random directions.  The step's tensors are rounded to bf16
    between its five stages, each off by 2^-8 of its values at most and independently: a few times 2^-8 of the root
    of the sum of the squares that the direction sees; eight holds them."""
    B, H, N, D = 1, 2, 90, 64
    axes = fa.RopeAxes(DIMS[D])
    q0, k0, v, wq, wk, pos, dout = _layer(B, H, N, D, seed=40)
    grads = _step(q0, k0, v, wq, wk, pos, dout, axes)[6:]
    grads = (grads[1], grads[2], grads[0], grads[3], grads[4])  # of q0, k0, v, wq, wk
    at = [x.double() for x in (q0, k0, v, wq, wk)]

    def loss(a):
        q, k = (ref.norm_rope(x, w, EPS, pos, DIMS[D], "adjacent") for x, w in ((a[0], a[3]), (a[1], a[4])))
        return (ref.attend(q, k, a[2], 1 / math.sqrt(D))[0] * dout.double()).sum()

    step = 2.0 ** -12
    for seed in range(3):
        d = [_rand(x.shape, 60 + 7 * seed + i, torch.float64) for i, x in enumerate(at)]
        moved = (loss([x + step * y for x, y in zip(at, d)]) - loss([x - step * y for x, y in zip(at, d)])) / (2 * step)
        along = sum((g.double() * y).sum() for g, y in zip(grads, d))
        size = math.sqrt(sum(float((g.double() * y).square().sum()) for g, y in zip(grads, d)))
        assert abs(float(moved - along)) <= 8 * 2.0 ** -8 * size


def test_a_captured_step_replays_with_new_inputs():
    B, H, N, D = 2, 2, 160, 128
    axes = fa.RopeAxes(DIMS[D])
    a, b = _layer(B, H, N, D, seed=1), _layer(B, H, N, D, seed=80)
    want = [x.clone() for x in _step(*b, axes, causal=True)]
    graph = torch.cuda.CUDAGraph()
    _step(*a, axes, causal=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = _step(*a, axes, causal=True)
    for x, y in zip(a, b):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(130, 257), (33, 5), (1, 129), (260, 128)])
def test_boolean_masks_at_any_byte(offset, D, Nq, Nk):
    B, H = 2, 2
    buf = torch.zeros(B * H * Nq * Nk + 8, dtype=torch.uint8, device="cuda")
    keep = buf[offset:offset + B * H * Nq * Nk].view(B, H, Nq, Nk)
    g = torch.Generator(device="cuda").manual_seed(5)
    kept = torch.rand(B, H, Nq, Nk, generator=g, device="cuda") < 0.7
    keep.copy_(kept * torch.randint(1, 256, (B, H, Nq, Nk), generator=g, device="cuda"))  # any nonzero byte
    buf[:offset], buf[offset + keep.numel():] = 255, 255                                  # (what lies around it)
    x = _inputs(B, H, H, Nq, Nk, D, full_mask=keep, dlse=True)
    _check_bwd(fa.bwd(**x), x)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(130, 256), (65, 4), (200, 131)])
def test_additive_masks_off_16_bytes(D, Nq, Nk):
    B, H = 1, 2
    buf = torch.full((B * H * Nq * Nk + 8,), math.nan, device="cuda")
    m = buf[1:1 + B * H * Nq * Nk].view(B, H, Nq, Nk)
    m.copy_(_rand((B, H, Nq, Nk), 4, torch.float32))
    m[..., ::5] = -math.inf
    x = _inputs(B, H, H, Nq, Nk, D, full_mask=m, causal=True, dlse=True)
    _check_bwd(fa.bwd(**x), x)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_gradient_of_lse_of_rows_that_see_nothing(bad):
    """LSE is -inf there, and its gradient often not a number: it reaches nothing."""
    B, H, Nq, Nk, D = 1, 2, 140, 200, 64
    keep = torch.ones(B, 1, Nq, Nk, dtype=torch.bool, device="cuda")
    keep[:, :, 50:60] = False
    x = _inputs(B, H, H, Nq, Nk, D, full_mask=keep, dlse=True)
    want = fa.bwd(**x)
    x["dlse"][:, :, 50:60] = bad
    assert all(torch.equal(a, b) for a, b in zip(fa.bwd(**x), want))


def test_two_masked_gradients_on_two_streams():
    B, H, N, D = 1, 2, 500, 64
    keep = torch.rand(B, H, N, N, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") < 0.5
    x = _inputs(B, H, H, N, N, D, full_mask=keep)
    y = _inputs(B, H, H, N, N, D, full_mask=~keep, seed=20)
    want = fa.bwd(**x) + fa.bwd(**y)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = fa.bwd(**x, stream=a) + fa.bwd(**y, stream=b)
    a.synchronize(), b.synchronize()
    assert all(torch.equal(u, w) for u, w in zip(got, want))


def _packed(B, heads, Nq, Nk, cuts, seed):
    """Sequences packed into one row (another offset for each head), some empty stretches."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shift = torch.randint(0, 200, (B, heads, 1, 1), generator=g, device="cuda")
    row = (torch.arange(Nq, device="cuda")[:, None] + shift) * cuts // (Nq + 200)
    key = (torch.arange(Nk, device="cuda")[None] + shift) * cuts // (Nk + 200)
    keep = row == key
    keep[:, :, Nq // 3:Nq // 3 + 300] = False
    return keep


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("B,Hq,Hk,Nq,Nk,per_head,causal", [
    (1, 2, 2, 1500, 1500, False, False), (1, 2, 1, 2100, 900, True, False), (2, 4, 1, 700, 1300, True, True),
    (1, 1, 1, 5000, 300, False, False), (1, 1, 1, 200, 4500, False, False), (1, 8, 8, 1300, 1300, True, True)])
def test_tiles_without_a_kept_pair(D, B, Hq, Hk, Nq, Nk, per_head, causal):
    """Tiles that a mask leaves empty are left out: at either end, in between, whole units, whole pieces of cut units."""
    x = _inputs(B, Hq, Hk, Nq, Nk, D, full_mask=_packed(B, Hq if per_head else 1, Nq, Nk, 7, 3), causal=causal, dlse=True)
    _check_bwd(fa.bwd(**x), x)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nk,keys", [(5000, (3, 4100)), (4500, (4400, 4500)), (300, (0, 1)), (1000, (0, 0))])
def test_key_tiles_without_a_key(D, Nk, keys):
    m = torch.full((2, Nk), -math.inf, device="cuda")
    m[:, keys[0]:keys[0] + 1] = 0.5
    m[0, keys[1]:] = -0.25
    m[1] = 0 if keys == (0, 0) else m[1]
    x = _inputs(2, 2, 1, 333, Nk, D, key_mask=m, dlse=True)
    _check_bwd(fa.bwd(**x), x)


def test_one_pair_of_a_million():
    keep = torch.zeros(1, 1, 1100, 1000, dtype=torch.bool, device="cuda")
    keep[0, 0, 1027, 513] = True
    x = _inputs(1, 2, 2, 1100, 1000, 64, full_mask=keep, dlse=True)
    dq, dk, dv = got = fa.bwd(**x)
    _check_bwd(got, x)
    assert int((dv != 0).any(-1).sum()) == 2 and torch.equal(dv[:, :, 513], x["dout"][:, :, 1027])  # P = 1


def _far(x, step):
    """x [B, H, N, D] with its tokens `step` elements apart, in a buffer that passes 2^31 elements."""
    B, H, N, D = x.shape
    buf = torch.empty(B * N * step, dtype=x.dtype, device="cuda")
    assert buf.numel() > 2 ** 31
    y = buf.as_strided((B, H, N, D), (N * step, D, step, 1))
    y.copy_(x)
    return y


def test_offsets_past_32_bits():
    B, H, N, D = 2, 2, 140, 64
    x = _inputs(B, H, H, N, N, D, causal=True, dlse=True)
    want = fa.bwd(**x)
    step = 2 ** 23
    far = dict(x, **{n: _far(x[n], step) for n in ("q", "dout")})
    dq = _far(torch.zeros_like(x["q"]), step)
    dk, dv = torch.empty_like(x["k"]), _far(torch.zeros_like(x["v"]), step)
    ws = torch.empty(fa.bwd_workspace_bytes(B, H, H, N, N, D), dtype=torch.uint8, device="cuda")
    fa.fa_bwd(far["dout"], far["q"], x["k"], x["v"], x["out"], x["lse"], dq, dk, dv, ws, causal=True,
              scale=x["scale"], dlse=x["dlse"])
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), want))
    axes, pos = fa.RopeAxes(DIMS[D]), torch.arange(3 * N, dtype=torch.int32, device="cuda").view(N, 3)
    w = 1 + 0.3 * _rand((D,), 4, torch.float32)
    far_out = _far(torch.zeros_like(x["q"]), step)
    fa.fa_norm_rope(far["q"], None, pos, axes, w, None, far_out, None)
    assert torch.equal(far_out, fa.norm_rope(x["q"], None, pos, axes, w)[0])
    got = fa.norm_rope_bwd(far["dout"], None, far["q"], None, pos, axes, w)
    assert all(torch.equal(a, b) for a, b in zip(got[::2], fa.norm_rope_bwd(x["dout"], None, x["q"], None, pos, axes,
                                                                            w)[::2]))


@pytest.mark.parametrize("kind,N", [("bool", 47000), ("add", 33100)])
def test_masks_past_32_bits(kind, N):
    """A mask that keeps everything (adds 0 everywhere) leaves the results as they are, bit for bit; one that leaves
    the last rows out by its last bytes does not touch the others' dQ."""
    q, k, v, do = (_rand((1, 1, N, 32), i) for i in range(4))
    out, lse = fa.fwd(q, k, v)
    want = fa.bwd(do, q, k, v, out, lse)
    m = torch.ones(1, 1, N, N, dtype=torch.bool, device="cuda") if kind == "bool" else torch.zeros(1, 1, N, N, device="cuda")
    assert m.numel() * m.element_size() > 2 ** 31
    got = fa.bwd(do, q, k, v, out, lse, full_mask=m)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    m[:, :, -200:] = False if kind == "bool" else -math.inf
    dq = fa.bwd(do, q, k, v, out, lse, full_mask=m)[0]
    assert torch.equal(dq[:, :, :-200], want[0][:, :, :-200]) and bool((dq[:, :, -200:] == 0).all())


CHILD = r'''
import sys, torch
sys.path.insert(0, ROOT)
import unet_fa_fwd_gb300 as fa
from tests.test_gpu_bwd import _check, _full_mask, _inputs, _key_mask
assert fa.debug_build(), "the debug library was not loaded"
torch.cuda.set_device(0)
for D in (32, 64, 128):
    for size, kw in [((1, 2, 2, 257, 300), {}), ((2, 4, 1, 1100, 700), dict(causal=True)), ((1, 1, 1, 2000, 90), {}),
                     ((2, 2, 2, 130, 77), dict(key_mask=_key_mask(2, 77, 3))),
                     ((1, 2, 2, 300, 200), dict(full_mask=_full_mask("bool", 1, 2, 300, 200, 4))),
                     ((1, 2, 1, 140, 260), dict(full_mask=_full_mask("add", 1, 1, 140, 260, 4)))]:
        x = _inputs(*size, D, dlse=True, **kw)
        got = fa.bwd(**x)
        torch.cuda.synchronize()
        st, rec = fa.read_device_status(), fa.debug_report()
        assert st == 0 and rec == [0] * 8, (D, size, st, rec)
        _check(got, x)
print("debug build: no violation")
'''


def test_debug_build_reports_no_violation():
    r = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT))], cwd=ROOT,
                       env=dict(os.environ, FA_DEBUG="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "no violation" in r.stdout
