"""A tile withheld from the attention's gradient, for every head size and kind of mask:
the waits run out, each CTA drains what it has in flight (an additive mask's copies
among it), the status word says so and the context stays usable."""
import math

import pytest
import torch

import unet_fa_fwd_gb300 as fa

from .test_gpu_bwd import _inputs, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)


def _mask(kind, N):
    if kind == "none":
        return {}
    if kind == "key":
        m = torch.zeros(1, N, device="cuda")
        m[:, -3:] = -math.inf
        return dict(key_mask=m)
    m = _rand((1, 4, N, N), 3, torch.float32)
    return dict(full_mask=m if kind == "add" else m > -2)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("kind,N", [("none", 900), ("key", 900), ("bool", 901), ("add", 900), ("add", 901)])
def test_withheld_tile(monkeypatch, D, kind, N):
    x = _inputs(1, 4, 4, N, N, D, **_mask(kind, N))
    want = fa.bwd(**x)
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0
    monkeypatch.setenv("FA_FAULT_INJECT", "stall")
    monkeypatch.setenv("FA_WAIT_TIMEOUT_MS", "100")
    fa.bwd(**x)
    torch.cuda.synchronize()
    assert fa.read_device_status() == fa.binding.FA_ERR_TIMEOUT
    monkeypatch.delenv("FA_FAULT_INJECT")
    monkeypatch.delenv("FA_WAIT_TIMEOUT_MS")
    assert all(torch.equal(a, b) for a, b in zip(fa.bwd(**x), want))
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0
