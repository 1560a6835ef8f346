"""Additive masks of more than 2^31 elements: one mask, and a head's own behind others."""
import math

import pytest
import torch

import unet_fa_fwd_gb300 as fa

from .test_gpu_bwd import _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0


@pytest.mark.parametrize("Nk", [46404, 46401])  # copied 16 bytes and 4 bytes at a time
def test_one_mask(Nk):
    """One that adds 0 everywhere leaves the results as they are, bit for bit; one that leaves the last rows out by
    its last elements does not touch the others' dQ."""
    N = 46404
    q, do = (_rand((1, 1, N, 32), i) for i in range(2))
    k, v = (_rand((1, 1, Nk, 32), i) for i in range(2, 4))
    out, lse = fa.fwd(q, k, v)
    want = fa.bwd(do, q, k, v, out, lse)
    m = torch.zeros(1, 1, N, Nk, device="cuda")
    assert m.numel() > 2 ** 31
    got = fa.bwd(do, q, k, v, out, lse, full_mask=m)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    m[:, :, -200:] = -math.inf
    dq = fa.bwd(do, q, k, v, out, lse, full_mask=m)[0]
    assert torch.equal(dq[:, :, :-200], want[0][:, :, :-200]) and bool((dq[:, :, -200:] == 0).all())
    # a large finite mask on these rows: their own sums, by the same offsets
    m[:, :, -200:] = -1e9
    low = lse.clone()
    low[:, :, -200:] -= 1e9
    dq = fa.bwd(do, q, k, v, out, low, full_mask=m)[0]
    assert torch.equal(dq[:, :, :-200], want[0][:, :, :-200])
    # (P within 2^-13 of itself either way: results of one bf16 rounding, P's and dS's, as in the tests of ordinary rows)
    a, b = dq[:, :, -200:].double(), want[0][:, :, -200:].double()
    assert float((a - b).norm()) <= 5e-3 * float(b.norm())


def test_a_heads_own_mask():
    """The last head's mask leaves out half of the keys; its gradients are those of the call on that head alone (whose
    units are cut elsewhere: sums in another order).  Sums that differ in their last bits may lie on either side of
    the middle between two bf16 numbers and come out a whole step apart: 2^-7 of 1 among 8-bit significands, so up to
    2^-7 of the value (2^-8, as this test first had it, is half a step).  P and dS are the same numbers on both sides
    and the sums fp32: the rest is far below 2^-10 of the largest."""
    H, N = 3, 27000
    q, k, v, do = (_rand((1, H, N, 32), i) for i in range(4))
    m = torch.zeros(1, H, N, N, device="cuda")
    assert m.numel() > 2 ** 31
    m[:, -1, :, ::2] = -math.inf
    one = [x[:, -1:].contiguous() for x in (do, q, k, v)]
    own = m[:, -1:].contiguous()
    out, lse = fa.fwd(q, k, v)
    out[:, -1:], lse[:, -1:] = fa.fwd_ex(*one[1:], full_mask=own)
    got = fa.bwd(do, q, k, v, out, lse, full_mask=m)
    want = fa.bwd(*one, out[:, -1:].contiguous(), lse[:, -1:].contiguous(), full_mask=own)
    assert bool((got[1][:, -1, ::2] == 0).all()) and bool((got[2][:, -1, ::2] == 0).all())
    for a, b in zip(got, want):
        a, b = a[:, -1:].double(), b.double()
        assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -10 * b.abs().max()).all())
