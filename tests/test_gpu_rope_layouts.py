"""Rotary positions in place, in slices of one buffer whatever the order of its axes: the same bits as
into new tensors, and nothing else of the buffer changes."""
import pytest
import torch

import unet_fa_fwd_gb300 as fa

pytestmark = pytest.mark.gpu

# order of (B, H, N) in memory, from the slowest
ORDERS = [("B", "N", "H"), ("B", "H", "N"), ("N", "B", "H"), ("H", "B", "N"), ("H", "N", "B"), ("N", "H", "B")]


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("D,dtype", [(64, torch.bfloat16), (32, torch.float32), (128, torch.float16)])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_in_place(order, D, dtype, pairing):
    size = dict(B=2, H=8, N=13)
    g = torch.Generator(device="cuda").manual_seed(1)
    buf = torch.randn(*(size[a] for a in order), D, generator=g, device="cuda").to(dtype)
    x = buf.permute(*(order.index(a) for a in "BHN"), 3)
    before = x.clone()
    q, k = x[:, :4], x[:, 4:6]
    pos = torch.randint(0, 500, (2, 13, 2), generator=g, device="cuda", dtype=torch.int32)
    axes = fa.RopeAxes((D // 2, D // 2))
    want = fa.rope(q, k, pos, axes, pairing=pairing)
    fa.fa_rope(q, k, pos, axes, q, k, pairing=pairing)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, 6:], before[:, 6:])
    # and back, from there into the buffer's other slices: k's gradient where v is
    fa.fa_rope(k, None, pos, axes, x[:, 6:], None, pairing=pairing, inverse=True)
    assert torch.equal(x[:, 6:], fa.rope_bwd(k, None, pos, axes, pairing=pairing)[0])
    assert torch.equal(x[:, 4:6], want[1])


def test_in_place_in_heads_of_q_k_and_v_together():
    """[B, N, H, 3, D]: the three lie side by side in each head."""
    g = torch.Generator(device="cuda").manual_seed(2)
    buf = torch.randn(2, 9, 4, 3, 64, generator=g, device="cuda").bfloat16()
    before = buf.clone()
    q, k = buf[:, :, :, 0].transpose(1, 2), buf[:, :, :, 1].transpose(1, 2)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")[:, None]
    axes = fa.RopeAxes((64,))
    want = fa.rope(q, k, pos, axes)
    fa.fa_rope(q, k, pos, axes, q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(buf[:, :, :, 2], before[:, :, :, 2])
    with pytest.raises(RuntimeError, match="INVALID_ARGUMENT"):
        fa.fa_rope(q, k, pos, axes, k, q)
