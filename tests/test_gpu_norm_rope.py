"""The norm of queries and keys with the rotary positions, and its gradient, on the
GPU against their 64-bit definitions.

Tolerances.  A row's sum of squares adds at most 16 terms in a thread and 5 joins,
so 1 / sqrt of it is within (21 / 2 + 4) 2^-24 < 2^-20 (rsqrtf: 2 units); a rotated
pair adds the rotation's 2^-21 and three roundings: an output is within
2^-19 (|a| + |b|) of its pair before it is rounded to its type.  The gradient of x
has two such factors more: 2^-18 of the sizes of its terms.  The gradients of the
weights add up to 100 values in a thread, 5 + 8 + 32 joins and 32 sums of a block's
rows: 2^-16 of the sizes of their terms.
"""
import pytest
import torch

import unet_fa_fwd_gb300 as fa

from . import grad_ref as ref

pytestmark = pytest.mark.gpu

DIMS = {128: (16, 56, 56), 64: (16, 24, 24), 32: (8, 12, 12)}
TYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)
    yield


def _rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _pos(shape, seed, lo=-70000, hi=70000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _near(got, want, size, part):
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + size * part
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half a step of its subnormals
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def _check_forward(y, x, w, pos, D, pairing, eps=EPS, **kw):
    want = ref.norm_rope(x, w, eps, pos, DIMS[D], pairing, **kw)
    _near(y, want, ref.pair_size(ref.norm(x, w, eps)[1], pairing), 2.0 ** -19)


def _check_backward(dx, dw, dy, x, w, pos, D, pairing, eps=EPS, **kw):
    want, dw_want, size, dw_size = ref.norm_rope_bwd(dy, x, w, eps, pos, DIMS[D], pairing, **kw)
    _near(dx, want, size, 2.0 ** -18)
    assert (dw is None) == (w is None)
    if dw is not None:
        assert dw.dtype == torch.float32
        _near(dw, dw_want, dw_size, 2.0 ** -16)


def _weights(kind, dtype, D):
    if kind == "none":
        return None, None
    w = [(1 + 0.3 * _rand((D,), torch.float32, s)).to(dtype if kind == "same" else torch.float32) for s in (5, 6)]
    return (w[0], None) if kind == "q" else (None, w[1]) if kind == "k" else tuple(w)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("weight,B,Hq,Hk,N", [("fp32", 1, 1, 1, 1), ("same", 2, 3, 1, 77), ("q", 3, 8, 2, 131),
                                             ("k", 1, 5, 3, 19), ("none", 2, 2, 2, 33)])
def test_against_definition(D, dtype, pairing, weight, B, Hq, Hk, N):
    axes = fa.RopeAxes(DIMS[D], theta=(256.0, 1e4, 5e5), scale=(1.0, 0.25, -1.5))
    kw = dict(theta=(256.0, 1e4, 5e5), scale=(1.0, 0.25, -1.5))
    x = _rand((B, N, Hq + 2 * Hk, D), dtype, 1)
    x[:, ::3] *= 30  # rows of unequal size
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    pos = _pos((B, N, 3), 2)
    wq, wk = _weights(weight, dtype, D)
    qo, ko = fa.norm_rope(q, k, pos, axes, wq, wk, eps=EPS, pairing=pairing)
    assert qo.is_contiguous() and qo.shape == q.shape and ko.shape == k.shape
    _check_forward(qo, q, wq, pos, D, pairing, **kw)
    _check_forward(ko, k, wk, pos, D, pairing, **kw)
    dqo, dko = _rand((B, Hq, N, D), dtype, 3), _rand((B, Hk, N, D), dtype, 4)
    dq, dk, dwq, dwk = fa.norm_rope_bwd(dqo, dko, q, k, pos, axes, wq, wk, eps=EPS, pairing=pairing, token_major=True)
    assert dq.transpose(1, 2).is_contiguous()
    _check_backward(dq, dwq, dqo, q, wq, pos, D, pairing, **kw)
    _check_backward(dk, dwk, dko, k, wk, pos, D, pairing, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_rows_off_16_bytes_shared_positions_q_alone(dtype, D, pairing):
    """Rows that start at odd elements are read one element at a time; [N, A] positions; no keys."""
    axes = fa.RopeAxes(DIMS[D])
    B, H, N = 2, 3, 45
    wide = _rand((B, H, N, D + 1), dtype, 1)
    q, dy = wide[..., 1:], _rand((B, H, N, D + 3), dtype, 2)[..., 3:]
    pos = _pos((N, 3), 3)
    w = 1 + 0.3 * _rand((D,), torch.float32, 4)
    y, none = fa.norm_rope(q, None, pos, axes, w, eps=EPS, pairing=pairing)
    assert none is None
    _check_forward(y, q, w, pos, D, pairing)
    dq, dk, dw, dwk = fa.norm_rope_bwd(dy, None, q, None, pos, axes, w, eps=EPS, pairing=pairing)
    assert dk is None and dwk is None
    _check_backward(dq, dw, dy, q, w, pos, D, pairing)


def test_odd_output_rows_and_what_lies_between_them():
    D, B, H, N = 64, 2, 2, 21
    axes = fa.RopeAxes(DIMS[D])
    q, dy, pos = _rand((B, H, N, D), torch.bfloat16, 1), _rand((B, H, N, D), torch.bfloat16, 2), _pos((B, N, 3), 3)
    for off in (1, 8):
        wide = torch.full((B, H, N, D + 2 * off), 7.0, dtype=torch.bfloat16, device="cuda")
        fa.fa_norm_rope(q, None, pos, axes, None, None, wide[..., off:off + D], None)
        _check_forward(wide[..., off:off + D], q, None, pos, D, "adjacent")
        assert bool((wide[..., :off] == 7).all()) and bool((wide[..., off + D:] == 7).all())
        wide.fill_(7.0)
        fa.fa_norm_rope_bwd(dy, None, q, None, pos, axes, None, None, wide[..., off:off + D], None, None, None, None)
        _check_backward(wide[..., off:off + D], None, dy, q, None, pos, D, "adjacent")
        assert bool((wide[..., :off] == 7).all()) and bool((wide[..., off + D:] == 7).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place(dtype):
    D, B, H, N = 128, 2, 5, 37
    axes = fa.RopeAxes(DIMS[D])
    x = _rand((B, N, 2 * H, D), dtype, 1)
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:].transpose(1, 2)
    pos, w = _pos((B, N, 3), 2), 1 + 0.3 * _rand((D,), dtype, 3)
    dqo, dko = _rand((B, H, N, D), dtype, 4), _rand((B, H, N, D), dtype, 5)
    want = fa.norm_rope(q, k, pos, axes, w, w)
    grads = fa.norm_rope_bwd(dqo, dko, q, k, pos, axes, w, w)
    ws = torch.empty(fa.norm_rope_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    dw = torch.empty(2, D, device="cuda")
    # gradients over the outputs' gradients (queries) and over the inputs (keys)
    k2 = x[:, :, H:].transpose(1, 2).clone()
    fa.fa_norm_rope_bwd(dqo, dko, q, k2, pos, axes, w, w, dqo, k2, dw[0], dw[1], ws)
    assert torch.equal(dqo, grads[0]) and torch.equal(k2, grads[1])
    assert torch.equal(dw[0], grads[2]) and torch.equal(dw[1], grads[3])
    fa.fa_norm_rope(q, k, pos, axes, w, w, q, k)  # slices of the projection, in place
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_rows_of_zeros_and_what_is_not_finite():
    """A row of zeros gives zeros and gradients of size 1 / sqrt(eps); NaN stays in its own row and the weights."""
    D, B, H, N = 64, 1, 2, 40
    axes = fa.RopeAxes(DIMS[D])
    q, dy, pos = _rand((B, H, N, D), torch.float32, 1), _rand((B, H, N, D), torch.float32, 2), _pos((B, N, 3), 3)
    w = 1 + 0.3 * _rand((D,), torch.float32, 4)
    q[0, 0, 3] = 0
    y, _ = fa.norm_rope(q, None, pos, axes, w, eps=1e-5)
    assert bool((y[0, 0, 3] == 0).all())
    dq, _, dw, _ = fa.norm_rope_bwd(dy, None, q, None, pos, axes, w, eps=1e-5)
    _check_backward(dq, dw, dy, q, w, pos, D, "adjacent", eps=1e-5)
    q[0, 1, 7, 5] = float("nan")
    bad, _ = fa.norm_rope(q, None, pos, axes, w, eps=1e-5)
    grad = fa.norm_rope_bwd(dy, None, q, None, pos, axes, w, eps=1e-5)
    for got, want in ((bad, y), (grad[0], dq)):
        same = (got == want).all(-1)
        assert not bool(same[0, 1, 7]) and int((~same).sum()) == 1 and bool(got[0, 1, 7].isnan().all())
    assert bool(grad[2].isnan().all())


def test_many_rows_repeat_bit_for_bit():
    """More token blocks than the grid holds (a block walks several) and head groups; the sums' order is fixed."""
    D, B, Hq, Hk, N = 32, 3, 7, 3, 30011
    axes = fa.RopeAxes(DIMS[D])
    q, k = _rand((B, Hq, N, D), torch.bfloat16, 1), _rand((B, Hk, N, D), torch.bfloat16, 2)
    dq, dk, pos = _rand((B, Hq, N, D), torch.bfloat16, 3), _rand((B, Hk, N, D), torch.bfloat16, 4), _pos((B, N, 3), 5)
    w = 1 + 0.3 * _rand((D,), torch.float32, 6)
    one = fa.norm_rope_bwd(dq, dk, q, k, pos, axes, w, w)
    two = fa.norm_rope_bwd(dq, dk, q, k, pos, axes, w, w)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    # 900000 rows over 304 blocks of 64 rows each: 50 values a thread, as the tolerance counts
    _check_backward(one[0], one[2], dq, q, w, pos, D, "adjacent")
    _check_backward(one[1], one[3], dk, k, w, pos, D, "adjacent")


def test_gradient_is_that_of_differences():
    """Directional differences of the forward in 32 bits (a step of 2^-7: the second order is 2^-14 of the values,
    their rounding 2^-24 / 2^-7)."""
    D, B, H, N = 64, 1, 2, 9
    axes = fa.RopeAxes(DIMS[D])
    q, dy, pos = _rand((B, H, N, D), torch.float32, 1), _rand((B, H, N, D), torch.float32, 2), _pos((B, N, 3), 3, 0, 90)
    w = 1 + 0.3 * _rand((D,), torch.float32, 4)
    dq, _, dw, _ = fa.norm_rope_bwd(dy, None, q, None, pos, axes, w)
    step = 2.0 ** -7
    for seed in range(3):
        v, vw = _rand(q.shape, torch.float32, 10 + seed), _rand((D,), torch.float32, 20 + seed)
        up = fa.norm_rope(q + step * v, None, pos, axes, w + step * vw)[0].double()
        down = fa.norm_rope(q - step * v, None, pos, axes, w - step * vw)[0].double()
        moved = ((up - down) * dy.double()).sum() / (2 * step)
        along = (dq.double() * v.double()).sum() + (dw.double() * vw.double()).sum()
        size = ((up - down).abs() * dy.double().abs()).sum() / (2 * step)
        assert abs(float(moved - along)) <= float(size) * 2.0 ** -12


def test_other_stream_and_graph():
    D, B, H, N = 128, 1, 4, 300
    axes = fa.RopeAxes(DIMS[D])
    q, dy, pos = _rand((B, H, N, D), torch.bfloat16, 1), _rand((B, H, N, D), torch.bfloat16, 2), _pos((B, N, 3), 3)
    w = 1 + 0.3 * _rand((D,), torch.float32, 4)
    want = fa.norm_rope(q, q, pos, axes, w, w) + fa.norm_rope_bwd(dy, dy, q, q, pos, axes, w, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fa.norm_rope(q, q, pos, axes, w, w, stream=side) + fa.norm_rope_bwd(dy, dy, q, q, pos, axes, w, w,
                                                                             stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.norm_rope(q, q, pos, axes, w, w) + fa.norm_rope_bwd(dy, dy, q, q, pos, axes, w, w)
    q.mul_(2.0).add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    want = fa.norm_rope(q, q, pos, axes, w, w) + fa.norm_rope_bwd(dy, dy, q, q, pos, axes, w, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
