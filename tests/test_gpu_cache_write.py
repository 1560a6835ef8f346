"""Writes whose first positions lie before the sequence: token i belongs at start + i, and the tokens
that have no place are not written."""
import pytest
import torch

import unet_fa_fwd_gb300 as fa
from unet_fa_fwd_gb300.binding import FA_ERR_INDEX

from . import cache_ref as ref
from .test_gpu_cache import _ints, _new, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)
    assert fa.read_device_status() == 0
    yield
    assert fa.read_device_status() == 0


@pytest.mark.parametrize("page", [32, 128])
@pytest.mark.parametrize("before", [1, 3, 40, 130])
def test_tokens_before_the_sequence_are_not_written(page, before):
    H, N, D = 2, 140, 64
    x, y = _rand((2, H, N, D), 1), _rand((2, H, N, D), 2)
    cache, table = _new(2, 300, H, page, D, 3, fill=0)
    fa.cache_write(cache, x, y, table, _ints([-before, 0]), _ints([N, N]))
    assert fa.read_device_status() == FA_ERR_INDEX
    held = N - before
    for got, new in zip(fa.cache_read(cache, table, _ints([held, N]), N), (x, y)):
        assert torch.equal(got[0, :, :held].double(), ref.quantised(new[0, :, before:], page)[0])
        assert torch.equal(got[1].double(), ref.quantised(new[1], page)[0])
    past = cache.k.view(torch.uint8)[table[0, held // page].long(), :, held % page:]
    assert not bool(past.any())  # rows behind the last token are as they were


@pytest.mark.parametrize("start,count", [(-8, 8), (-9, 8), (-2 ** 31, 8), (-1, 0), (-1, 1)])
def test_nothing_has_a_place(start, count):
    x = _rand((1, 1, 8, 32), 4)
    cache, table = _new(1, 64, 1, 32, 32, 5, fill=0)
    fa.cache_write(cache, x, x, table, _ints([start]), _ints([count]))
    assert fa.read_device_status() == FA_ERR_INDEX
    assert not bool(cache.k.view(torch.uint8).any()) and not bool(cache.k_scale.view(torch.uint8).any())
