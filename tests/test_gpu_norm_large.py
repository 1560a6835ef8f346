"""Rows whose squares sum past fp32's range: the norm with rotary positions makes zeros of
them, and their gradients are zeros, also where the sum of dy w x is past the range too."""
import pytest
import torch

import unet_fa_fwd_gb300 as fa

from .test_gpu_norm_rope import DIMS, _pos, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("size", [1e20, 1e38])
def test_rows_past_the_range(dtype, D, pairing, size):
    B, H, N = 2, 3, 50
    axes = fa.RopeAxes(DIMS[D])
    q, dy, pos = _rand((B, H, N, D), dtype, 1), _rand((B, H, N, D), dtype, 2).abs() + 1, _pos((B, N, 3), 3)
    w = 1 + 0.3 * _rand((D,), torch.float32, 4).abs()
    rows = (slice(None), slice(None), slice(7, 20))
    small = q.clone()
    small[rows] = 0                       # (with eps such a row has no dw either)
    q[rows] = size
    y, _ = fa.norm_rope(q, None, pos, axes, w, pairing=pairing)
    assert bool((y[rows] == 0).all())
    dq, _, dw, _ = fa.norm_rope_bwd(dy, None, q, None, pos, axes, w, pairing=pairing)
    want, _, dw_want, _ = fa.norm_rope_bwd(dy, None, small, None, pos, axes, w, pairing=pairing)
    assert bool((dq[rows] == 0).all()) and bool(dq.isfinite().all())
    want[rows] = 0
    assert torch.equal(dq, want) and torch.equal(dw, dw_want)
