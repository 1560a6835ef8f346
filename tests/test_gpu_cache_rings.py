"""The cached attention where a CTA walks many tiles: its rings come round
several times, and it goes from one unit to the next with its slots in use.
Every head has scales of its own, powers of four apart, so that another tile's
scale shows.  Definitions and tolerances as in test_gpu_cache.py.
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


def _filled(lens, H, page, D, seed):
    """A cache of sequences whose K and V have a size of their own in each sequence and head (V: powers
    of four from 4^-3 to 4^3; K: from 4^-2 to 4^2, other ones in every second tile), and the values it
    holds.  The first two tiles' keys point the queries' way (dimension 0), so that they weigh as much
    as the rest."""
    B, N = len(lens), max(lens)
    cache, table = _new(B, N, H, page, D, seed)
    k, v = _rand((B, H, N, D), seed + 1).float(), _rand((B, H, N, D), seed + 2).float()
    g = torch.Generator(device="cuda").manual_seed(seed + 3)
    size = lambda n: torch.exp2(2.0 * torch.randint(-n, n + 1, (B, H, 1, 1), generator=g, device="cuda"))  # noqa: E731
    v = v * size(3)
    odd = torch.arange(N, device="cuda")[:, None] // 128 % 2 == 1
    k = k * torch.where(odd, size(2), size(2))
    k[:, :, :256, 0] = k[:, :, :256].abs().amax((2, 3))[..., None]
    fa.cache_write(cache, k.to(BF16), v.to(BF16), table, _ints([0] * B), _ints(lens))
    ks, vs = fa.cache_read(cache, table, _ints(lens), N)
    return cache, table, [ks[b, :, :n] for b, n in enumerate(lens)], [vs[b, :, :n] for b, n in enumerate(lens)]


def _queries(shape, ks, seed):
    """Rows whose scores (scale 1 / sqrt D) are a few units, whatever the size of their keys: the size
    of a row is that of the head's first tile of keys, which they point to."""
    q = _rand(shape, seed).float()
    B, Hq = shape[:2]
    for b in range(B):
        first = ks[b][:, :128].float().abs().amax((1, 2)).repeat_interleave(Hq // ks[b].shape[0])
        q[b] *= (2.0 / first)[:, None, None]
        q[b, ..., 0] = (3.0 * math.sqrt(shape[-1]) / first)[:, None]
    return q.to(BF16)


def _check(q, cache, table, lens, ks, vs, causal, rows=None, seqs=None):
    """Against the definition, at the rows (slices) and sequences given, and twice for equal bits."""
    Hq, Nq, D = q.shape[1:]
    out, lse = fa.fwd_cache(q, cache, table, _ints(lens), causal=causal)
    again = fa.fwd_cache(q, cache, table, _ints(lens), causal=causal)
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    for b in range(len(lens)) if seqs is None else seqs:
        g = Hq // ks[b].shape[0]
        for h in range(ks[b].shape[0]):  # a head at a time: the definition keeps every score
            of = slice(h * g, h * g + g)
            for lo, hi in rows or ((0, Nq),):
                want = ref.attend(q[b, of, lo:hi], ks[b][h:h + 1], vs[b][h:h + 1], D ** -0.5, causal,
                                  lens[b] - Nq + lo)
                _close(out[b, of, lo:hi], lse[b, of, lo:hi], want, vs[b][h:h + 1], cache.k.shape[2],
                       (b, h, lo, lens[b]), g * Nq <= 16)


@pytest.mark.parametrize("D,page", [(128, 128), (128, 32), (64, 64), (32, 32)])
@pytest.mark.parametrize("causal", [False, True])
def test_last_row_tile_half_empty(D, page, causal):
    """300 rows of 24 heads on 16896 keys: one row tile of 256 and one of 44, some 40 tiles a CTA."""
    cache, table, ks, vs = _filled([16896], 24, page, D, 200)
    _check(_queries((1, 24, 300, D), ks, 201), cache, table, [16896], ks, vs, causal)


def test_many_row_tiles_the_last_half_empty():
    """2100 rows of 24 heads on 16896 keys, the first rows of each head and the last."""
    cache, table, ks, vs = _filled([16896], 24, 128, 128, 210)
    _check(_queries((1, 24, 2100, 128), ks, 211), cache, table, [16896], ks, vs, True, rows=((0, 300), (2000, 2100)))


def test_a_prompt_that_attends_to_itself():
    """10800 rows of 24 heads on 10800 keys: the rows around the first row tiles, and the last."""
    cache, table, ks, vs = _filled([10800], 24, 64, 128, 220)
    _check(_queries((1, 24, 10800, 128), ks, 221), cache, table, [10800], ks, vs, True,
           rows=((0, 260), (380, 400), (10700, 10800)))


def test_grouped_heads_with_a_half_empty_row_tile():
    """75 positions of 4 query heads to a key head (300 rows), 8 sequences of 8192 keys."""
    cache, table, ks, vs = _filled([8192] * 8, 8, 64, 64, 230)
    _check(_queries((8, 32, 75, 64), ks, 231), cache, table, [8192] * 8, ks, vs, True, seqs=(0, 3, 4, 7))


@pytest.mark.parametrize("D,page", [(128, 128), (64, 32)])
@pytest.mark.parametrize("causal", [False, True])
def test_runs_of_one_tile_units(D, page, causal):
    """20 rows: 24 units of one tile in a row, then 8 of six tiles, 120 times."""
    lens = ([100, 128, 77] + [700]) * 120
    cache, table, ks, vs = _filled(lens, 8, page, D, 240)
    _check(_queries((len(lens), 8, 20, D), ks, 241), cache, table, lens, ks, vs, causal, seqs=range(3, 480, 16))


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("rows,L,H", [(1, 119056, 24), (16, 119056, 24), (128, 38000, 24), (256, 38000, 24)])
def test_every_ring_comes_round(D, rows, L, H):
    """At least 35 tiles a CTA in each kernel."""
    cache, table, ks, vs = _filled([L], H, 128 if D == 64 else 64, D, 250)
    _check(_queries((1, H, rows, D), ks, 251), cache, table, [L], ks, vs, False)
