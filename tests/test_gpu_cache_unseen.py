"""What a row of the cached attention does not see does not reach it: numbers in
V that are not finite (0 times NaN is NaN on the tensor cores), and scales of
pages past the row's last key.

A row is a function of q and of the keys that it sees.  Two caches that agree
on those, page for page, give it the same bits: the other keys' probabilities
are exact zeros, and every unit that results are held in follows from what the
row sees.
"""
import math

import pytest
import torch

import unet_fa_fwd_gb300 as fa

from . import cache_ref as ref
from .test_gpu_cache import BF16, _close, _ints, _new, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)
    assert fa.read_device_status() == 0
    yield
    assert fa.read_device_status() == 0


# rows of a key head: few (4, 8, 16), pairs of key tiles, two row tiles, several units
SHAPES = [(1, 4), (2, 4), (3, 5), (1, 30), (4, 30), (1, 200), (1, 300), (2, 290)]


def _filled(k, v, page):
    """A cache holding k, v [1, H, L, D]."""
    L = k.shape[2]
    cache, table = _new(1, L, k.shape[1], page, k.shape[3], 300)
    fa.cache_write(cache, k, v, table, _ints([0]))
    return cache, table


def _rows(L, Nq, edge):
    """Rows (causal, at the end of L keys) that see nothing from key `edge` on, and those that do."""
    cut = min(max(edge - (L - Nq), 0), Nq)
    assert 0 < cut < Nq
    return slice(0, cut), slice(cut, Nq)


@pytest.mark.parametrize("D,page", [(32, 32), (64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("g,Nq", SHAPES)
@pytest.mark.parametrize("where", ["tile", "next tile"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_value_that_is_not_finite(D, page, g, Nq, where, value):
    """One channel of V at key `edge`, inside a tile or its first key: the rows before it keep their
    bits, those that see it give NaN in that channel, and no LSE changes.  (A tile's first key: so many
    heads that a CTA walks the tile with the one before it.)"""
    H, edge = (2, 384 + 77) if where == "tile" else (700 if g * Nq <= 16 else 160, 384)
    L = edge + (Nq + 1) // 2
    q, k, v = _rand((1, H * g, Nq, D), 301), _rand((1, H, L, D), 302), _rand((1, H, L, D), 303)
    bad = torch.arange(H, device="cuda") % 2 == 1  # in every second key head
    v[0, bad, edge, D - 3] = 0.0
    cache, table = _filled(k, v, page)
    want, lse = fa.fwd_cache(q, cache, table, _ints([L]), causal=True)
    v[0, bad, edge, D - 3] = value
    cache, table = _filled(k, v, page)
    out, got = fa.fwd_cache(q, cache, table, _ints([L]), causal=True)
    before, after = _rows(L, Nq, edge)
    bad = bad.repeat_interleave(g)
    assert torch.equal(out[0, ~bad], want[0, ~bad]) and torch.equal(got, lse)
    assert torch.equal(out[0, bad][:, before], want[0, bad][:, before])
    assert bool(out[0, bad][:, after, D - 3].isnan().all())


@pytest.mark.parametrize("g,Nq", SHAPES)
@pytest.mark.parametrize("far", [False, True])
def test_values_that_are_not_finite_before_every_row(g, Nq, far):
    """A NaN that all rows see reaches all of them in its channel (and none of the other channels,
    where its tile is seen whole); also where its tile's scores lie so far below the others that
    fp32 holds its weights as 0."""
    q, k, v = _rand((1, g, Nq, 64), 304), _rand((1, 1, 700, 64), 305), _rand((1, 1, 700, 64), 306)
    v[0, 0, 130, 5] = math.nan
    if far:  # scores of -400
        q[..., 0], k[:, :, 128:256, 0] = 8.0, -400.0
    cache, table = _filled(k, v, 64)
    out, lse = fa.fwd_cache(q, cache, table, _ints([700]), causal=True)
    bad = out.isnan()
    assert bool(bad[..., 5].all()) and int(bad.sum()) == g * Nq and bool(lse.isfinite().all())


@pytest.mark.parametrize("g,Nq", SHAPES)
@pytest.mark.parametrize("page", [32, 128])
def test_rows_that_see_no_key(g, Nq, page):
    """Rows before the first key, with NaN in every V: O = 0 and LSE = -inf."""
    q, k, v = _rand((1, g, Nq, 64), 307), _rand((1, 1, 300, 64), 308), _rand((1, 1, 300, 64), 309)
    v[...] = math.nan
    none = Nq // 2
    cache, table = _filled(k, v, page)
    for start in (-none, -Nq):
        gone = min(-start, Nq)
        out, lse = fa.fwd_cache(q, cache, table, _ints([300]), causal=True, q_start=_ints([start]))
        assert not bool(out[:, :, :gone].any()) and bool(torch.isneginf(lse[:, :, :gone]).all())
        assert bool(out[:, :, gone:].isnan().all()) and bool(lse[:, :, gone:].isfinite().all())
    out, lse = fa.fwd_cache(q, cache, table, _ints([0]), causal=True)
    assert not bool(out.any()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("D,page", [(32, 32), (64, 32), (64, 64), (128, 32)])
@pytest.mark.parametrize("g,Nq", SHAPES)
@pytest.mark.parametrize("where", ["tile", "next tile"])
@pytest.mark.parametrize("least,most", [(0, 30), (-100, 110)])
def test_scales_of_pages_that_are_not_seen(D, page, g, Nq, where, least, most):
    """V is 2^least before key `edge` (the first of a page, inside a tile or opening one) and 2^most times
    that from it on: the rows before it keep their bits, and are as exact as the pages that they see
    allow.  K's size changes by 2^40 there too."""
    H, edge = (2, 384 + 64) if where == "tile" else (700 if g * Nq <= 16 else 160, 384)
    L = edge + (Nq + 1) // 2
    q, k, v = _rand((1, H * g, Nq, D), 310), _rand((1, H, L, D), 311), _rand((1, H, L, D), 312)
    v *= 2.0 ** least
    cache, table = _filled(k, v, page)
    want, lse = fa.fwd_cache(q, cache, table, _ints([L]), causal=True)
    for _ in range(2):
        v[:, :, edge:] *= 2.0 ** ((most - least) / 2)
    k[:, :, edge:] *= 2.0 ** 40
    cache, table = _filled(k, v, page)
    out, got = fa.fwd_cache(q, cache, table, _ints([L]), causal=True)
    before, _ = _rows(L, Nq, edge)
    assert torch.equal(out[:, :, before], want[:, :, before]) and torch.equal(got[:, :, before], lse[:, :, before])
    ks, vs = (x[0, :2, :edge] for x in fa.cache_read(cache, table, _ints([L]), L))
    exact = ref.attend(q[0, :2 * g, before], ks, vs, D ** -0.5, True, L - Nq)
    _close(out[0, :2 * g, before], got[0, :2 * g, before], exact, vs, page, "", g * Nq <= 16)


@pytest.mark.parametrize("g,Nq", SHAPES)
@pytest.mark.parametrize("page", [32, 64, 128])
def test_scales_that_grow_along_the_diagonal(g, Nq, page):
    """Pages whose V grows by 2^8 for every 32 tokens: each row against the definition on the keys that
    it sees, with the error that the pages which it sees allow."""
    L, D = 700, 64
    q, k, v = _rand((1, g, Nq, D), 313), _rand((1, 1, L, D), 314), _rand((1, 1, L, D), 315)
    v *= torch.exp2(torch.arange(L, device="cuda") // page * (page / 4.0) - 88)[:, None]
    cache, table = _filled(k, v, page)
    out, lse = fa.fwd_cache(q, cache, table, _ints([L]), causal=True)
    ks, vs = (x[0] for x in fa.cache_read(cache, table, _ints([L]), L))
    for i in range(Nq):
        n = L - Nq + i + 1
        exact = ref.attend(q[0, :, i:i + 1], ks[:, :n], vs[:, :n], D ** -0.5)
        _close(out[0, :, i:i + 1], lse[0, :, i:i + 1], exact, vs[:, :n], page, i, g * Nq <= 16)


@pytest.mark.parametrize("g,Nq", SHAPES)
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_padded_rows_of_q_that_see_no_key(g, Nq, value):
    """Rows of q that are not finite (padding) and see nothing: O = 0 and LSE = -inf, as any row without
    keys; in an empty sequence too."""
    q, k, v = _rand((2, g, Nq, 64), 316), _rand((1, 1, 300, 64), 317), _rand((1, 1, 300, 64), 318)
    cache, table = _filled(k, v, 64)
    table = table.repeat(2, 1)
    none = Nq // 2
    ks, vs = (x[0] for x in fa.cache_read(cache, table[:1].contiguous(), _ints([300]), 300))
    want = ref.attend(q[0, :, none:], ks, vs, 0.125, True, 0)
    q[0, :, :none] = value
    q[1] = value
    out, lse = fa.fwd_cache(q, cache, table, _ints([300, 0]), causal=True, q_start=_ints([-none, 0]))
    for x, gone in ((0, slice(0, none)), (1, slice(0, Nq))):
        assert not bool(out[x, :, gone].any()) and bool(torch.isneginf(lse[x, :, gone]).all())
    _close(out[0, :, none:], lse[0, :, none:], want, vs, 64, "", g * Nq <= 16)
