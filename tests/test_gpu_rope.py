"""Rotary positions on the GPU against their 64-bit definition.

Tolerance: an output x0 c - x1 s is computed in fp32 from a cosine and a sine
that are each within 2^-22 of the true ones (the phase is exact to 2^-31 turns
at most, sincospif to 2 units of 2^-24), with three roundings of 2^-24, and
rounded once to its type: |error| <= eps/2 |y| + (|x0| + |x1|) 2^-21.
"""
import math

import pytest
import torch

import unet_fa_fwd_gb300 as fa

from . import cache_ref as ref

pytestmark = pytest.mark.gpu

DIMS = {128: (16, 56, 56), 64: (16, 24, 24), 32: (8, 12, 12)}


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)
    yield


def _rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _pos(shape, hi, seed, lo=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _check(got, x, want, pairing):
    D = x.shape[-1]
    a = x.double().abs()
    if pairing == "adjacent":
        size = a.unflatten(-1, (D // 2, 2)).sum(-1).repeat_interleave(2, -1)
    else:
        size = (a[..., :D // 2] + a[..., D // 2:]).repeat(1, 1, 1, 2)
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + size * 2.0 ** -21
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half a step of its subnormals
    err = (got.double() - want).abs()
    assert got.dtype == x.dtype and bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("B,Hq,Hk,N", [(1, 1, 1, 1), (2, 3, 1, 77), (3, 8, 2, 130)])
def test_rope_against_definition(D, dtype, pairing, B, Hq, Hk, N):
    axes = fa.RopeAxes(DIMS[D], theta=(256.0, 1e4, 5e5), scale=(1.0, 0.25, -1.5))
    x = _rand((B, N, Hq + 2 * Hk, D), dtype, 1)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)  # slices of a projection
    pos = _pos((B, N, 3), 5000, 2, -100)
    for inverse in (False, True):
        got = fa.rope(q, k, pos, axes, pairing=pairing, inverse=inverse, token_major=inverse)
        for y, z in zip(got, (q, k)):
            assert y.shape == z.shape and (y if not inverse else y.transpose(1, 2)).is_contiguous()
            _check(y, z, ref.rope(z, pos, DIMS[D], axes.theta, axes.scale, pairing, inverse), pairing)


def test_positions_of_any_size():
    """The reduction is exact: the far ends of int32 on every axis, and position 0 changes nothing."""
    far = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1, -1, 2 ** 30 + 12345, 119056], dtype=torch.int32, device="cuda")
    pos = torch.stack([far, far.flip(0), far.roll(2)], -1)
    pos[2] = 0
    x = _rand((1, 2, len(far), 128), torch.float32, 3)
    q, _ = fa.rope(x, None, pos, fa.RopeAxes(DIMS[128]))
    assert torch.equal(q[:, :, 2], x[:, :, 2])
    # Angles of 2^31 in 64 bits: pow is within 2^-52 and the product 2^-53 (2^31 * 1.5 * 2^-52 < 2^-20);
    # the kernel's turns are pow, the rounded 1 / (2 pi) and their product (2^31 * 2 * 2^-52 = 2^-20).
    want = ref.rope(x, pos, DIMS[128])
    err = (q.double() - want).abs()
    size = x.double().abs().unflatten(-1, (64, 2)).sum(-1).repeat_interleave(2, -1)
    assert bool((err <= want.abs() * 2.0 ** -24 + size * (2.0 ** -21 + 2.0 ** -19)).all()), float(err.max())


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_unaligned_rows(pairing):
    """Rows that do not start 16-byte aligned, in and out."""
    buf = _rand((2 * 3 * 40 * 65 + 9,), torch.bfloat16, 4)
    q = buf[1:1 + 2 * 3 * 40 * 65].view(2, 3, 40, 65)[..., :64]
    pos = _pos((40, 3), 300, 5)
    axes = fa.RopeAxes(DIMS[64])
    out = torch.full((2, 3, 40, 67), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_rope(q, None, pos, axes, out[..., 1:65], None, pairing=pairing)
    _check(out[..., 1:65], q, ref.rope(q, pos, DIMS[64], pairing=pairing), pairing)
    assert bool((out[..., 0] == 7).all()) and bool((out[..., 65:] == 7).all())
    # the same from aligned copies, bit for bit
    assert torch.equal(out[..., 1:65], fa.rope(q.contiguous(), None, pos, axes, pairing=pairing)[0])


def test_in_place_in_a_packed_projection():
    x = _rand((2, 50, 8, 64), torch.bfloat16, 6)
    before = x.clone()
    q, k = x[:, :, :4].transpose(1, 2), x[:, :, 4:6].transpose(1, 2)
    pos, axes = _pos((2, 50, 3), 90, 7), fa.RopeAxes(DIMS[64])
    want = fa.rope(q, k, pos, axes)
    fa.fa_rope(q, k, pos, axes, q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, :, 6:], before[:, :, 6:])


def test_broadcast_input_and_shared_positions():
    x = _rand((1, 1, 33, 32), torch.float16, 8)
    pos = _pos((33, 3), 64, 9)
    axes = fa.RopeAxes(DIMS[32])
    q, k = fa.rope(x.expand(4, 5, 33, 32), x.expand(4, 2, 33, 32), pos, axes)
    one = fa.rope(x, None, pos.expand(1, 33, 3), axes)[0]
    assert torch.equal(q, one.expand_as(q)) and torch.equal(k, one.expand_as(k))


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_gradient(pairing):
    """Against the formula, and against central differences of the 64-bit definition."""
    B, Hq, Hk, N, D = 2, 4, 2, 21, 64
    pos, axes = _pos((B, N, 3), 700, 10), fa.RopeAxes(DIMS[D], theta=256.0)
    dq, dk = _rand((B, Hq, N, D), torch.float32, 11), _rand((B, Hk, N, D), torch.float32, 12)
    gq, gk = fa.rope_bwd(dq, dk, pos, axes, pairing=pairing, token_major=True)
    for g, d in ((gq, dq), (gk, dk)):
        assert g.transpose(1, 2).is_contiguous()
        _check(g, d, ref.rope(d, pos, DIMS[D], 256.0, 1.0, pairing, True), pairing)
    x = _rand((B, Hq, N, D), torch.float64, 13)
    step = _rand((B, Hq, N, D), torch.float64, 14)
    f = lambda y: float((ref.rope(y, pos, DIMS[D], 256.0, 1.0, pairing) * dq.double()).sum())  # noqa: E731
    slope = (f(x + step) - f(x - step)) / 2  # the rotation is linear
    terms = (gq.double() * step)
    # each term of the sum is off by 2^-20 of |gradient| + |neighbours| at most
    assert abs(float(terms.sum()) - slope) <= 2.0 ** -19 * float(terms.abs().sum() + (dq.double() * step).abs().sum())


def test_gradient_into_a_packed_buffer():
    """dq, dk, dv of one token-major projection share a buffer."""
    d = torch.zeros(2, 30, 8, 64, device="cuda")
    dq, dk = _rand((2, 4, 30, 64), torch.float32, 15), _rand((2, 2, 30, 64), torch.float32, 16)
    pos, axes = _pos((30, 3), 90, 17), fa.RopeAxes(DIMS[64])
    fa.fa_rope(dq, dk, pos, axes, d[:, :, :4].transpose(1, 2), d[:, :, 4:6].transpose(1, 2), inverse=True)
    gq, gk = fa.rope_bwd(dq, dk, pos, axes)
    assert torch.equal(d[:, :, :4].transpose(1, 2), gq) and torch.equal(d[:, :, 4:6].transpose(1, 2), gk)
    assert not bool(d[:, :, 6:].any())


def test_other_stream_and_graph():
    pos, axes = _pos((2, 64, 3), 90, 18), fa.RopeAxes(DIMS[128])
    q, k = _rand((2, 4, 64, 128), torch.bfloat16, 19), _rand((2, 4, 64, 128), torch.bfloat16, 20)
    want = fa.rope(q, k, pos, axes)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.rope(q, k, pos, axes, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fa.rope(q, k, pos, axes)
    q.copy_(q.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], fa.rope(q, k, pos, axes)[0])


def test_rows_past_32_bit_offsets():
    """Strides that put the last rows past 2^31 elements."""
    buf = torch.empty((1 << 31) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    x = _rand((2, 3, 5, 128), torch.bfloat16, 21)
    q = torch.as_strided(buf, (2, 3, 5, 128), ((1 << 31) + 4096, 640, 128, 1))
    q.copy_(x)
    pos, axes = _pos((5, 3), 90, 22), fa.RopeAxes(DIMS[128])
    want = fa.rope(x, None, pos, axes)[0]
    assert torch.equal(fa.rope(q, None, pos, axes)[0], want)
    out = torch.as_strided(buf, (2, 3, 5, 128), ((1 << 31) + 4096, 640, 128, 1), 8192)
    fa.fa_rope(x, None, pos, axes, out, None)
    assert torch.equal(out, want)


def test_refusals():
    x = _rand((1, 2, 8, 64), torch.bfloat16, 23)
    pos, axes = _pos((8, 3), 9, 24), fa.RopeAxes(DIMS[64])
    with pytest.raises(ValueError, match="shape"):
        fa.rope(x, None, pos[:7], axes)
    with pytest.raises(TypeError, match="int32"):
        fa.rope(x, None, pos.long(), axes)
    with pytest.raises(TypeError, match="k must be"):
        fa.rope(x, x.float(), pos, axes)
    with pytest.raises(TypeError, match="bf16"):
        fa.rope(x.double(), None, pos, axes)
    with pytest.raises(ValueError, match="pairing"):
        fa.rope(x, None, pos, axes, pairing="odd")
    with pytest.raises(ValueError, match="last axis"):
        fa.rope(x.transpose(2, 3).contiguous().transpose(2, 3), None, pos, axes)
    with pytest.raises(ValueError, match="together"):
        fa.fa_rope(x, x, pos, axes, x, None)
    with pytest.raises(ValueError, match="must be on|CUDA"):
        fa.rope(x, None, pos.cpu(), axes)
    with pytest.raises(RuntimeError, match="INVALID_ARGUMENT"):
        fa.rope(x, None, pos, fa.RopeAxes((16, 24, 26)))
    with pytest.raises(RuntimeError, match="INVALID_ARGUMENT"):
        fa.fa_rope(x, None, pos, axes, x[:, :1].expand(1, 2, 8, 64), None)
    assert math.isfinite(float(x.float().sum()))
