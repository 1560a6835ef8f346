"""Gradients of the norm's weights over many rows: sums of one call against those of many
short ones, added up in 64 bits.  The terms are the same, so what differs is rounding in
the sums.

Terms of either sign: an addition is off by u / sqrt(3) of the sum so far in the mean
square (u = 2^-24, half a step), and one chain of m terms by sqrt(m / 2) u / sqrt(3) of the
result's norm.  A thread adds 32 heads in a row and keeps what later additions round off
(2.3 u); 5 + 3 joins by twos are sqrt(8) u / sqrt(3) = 1.6 u, a block's row and the result
0.8 u: 3 u together.  Both sides are such sums: 4.2 u, and 6 u = 2^-21.4 holds it.  One chain
a thread would be off by 14 u here and more.
"""
import pytest
import torch

import unet_fa_fwd_gb300 as fa

from .test_gpu_norm_rope import DIMS, TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype,D,H,N,pairing", [
    (TYPES[2], 128, 24, 120000, "adjacent"), (TYPES[2], 128, 3, 700000, "halves"), (TYPES[0], 64, 24, 400000, "halves"),
    (TYPES[1], 32, 40, 400000, "adjacent")])
def test_weights_gradients_over_many_rows(dtype, D, H, N, pairing):
    g = torch.Generator(device="cuda").manual_seed(N)
    q, dy = (torch.empty(1, H, N, D, dtype=dtype, device="cuda") for _ in range(2))
    for h in range(H):
        for x in (q, dy):
            x[:, h].copy_(torch.randn(N, D, generator=g, device="cuda"))
    pos = torch.randint(0, 5000, (N, 3), generator=g, device="cuda", dtype=torch.int32)
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    axes = fa.RopeAxes(DIMS[D])
    got = fa.norm_rope_bwd(dy, None, q, None, pos, axes, w, pairing=pairing)[2]
    want = torch.zeros(D, dtype=torch.float64, device="cuda")
    step = 1000
    for n in range(0, N, step):
        s = slice(n, n + step)
        want += fa.norm_rope_bwd(dy[:, :, s], None, q[:, :, s], None, pos[s], axes, w, pairing=pairing)[2].double()
    assert float((got.double() - want).norm()) <= 6 * 2.0 ** -24 * float(want.norm())
