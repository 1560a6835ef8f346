"""The paged e4m3 cache and the attention to it on the GPU, against 64-bit
definitions (tests/cache_ref.py).

Attention tolerance.  With A = sum_j p_j |v_j| (a row's mean of |v|),
Q = max_j sum_d |scale q_d k_jd| and Q' = max_j |scale| max_d |q_d| sum_d |k_jd|:
  * scores: the codes are exact.  q is held in two e4m3 numbers, the row's
    largest element at 224 or more; the second's least step (2^-9 for many
    rows, where it has the first's scale) leaves 2^-10 / 224 < 2^-17.8 of the
    largest element: 2^-17.8 Q'.  The tensor cores' fp32 sums are within 2^-19
    of the sum of magnitudes (2^-18 Q with the two parts), and 2^-22 |t| for the
    fp32 products and 2^-22 for ex2: together
    dt <= 2^-17 Q + 2^-17.8 Q' + 2^-21 moves every p by that factor and LSE by dt;
  * p is held in 12 bits (up to 16 rows of a key head) or in f16 (half a step:
    2^-11), so sum p v moves by at most 2^-11 A;
  * the 12 bits end at e4m3's subnormals: with the row's largest p at 2^7 or
    more, the third column's least step 2^-9 stands for 2^-17, so a p is off by
    half of that, 2^-25 of the largest; f16's end at 2^-24, the row's largest p
    being 1 or more.  O moves by 2^-25 |v_j| a key, times the ratio of the
    largest scale of V to the page's own, among the 128-key tile's pages with
    few rows, among the sequence's with many (weight): F in all;
  * fp32 sums over N keys, a 32-key step at a time: (N / 32) 2^-24 A;
  * O is rounded once to bf16: 2^-8 |O|.
"""
import math
import os
import subprocess
import sys

import pytest
import torch

import unet_fa_fwd_gb300 as fa
from unet_fa_fwd_gb300.binding import FA_ERR_INDEX, FA_ERR_TIMEOUT

from . import cache_ref as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.load_library()
    torch.cuda.set_device(0)
    assert fa.read_device_status() == 0
    yield
    assert fa.read_device_status() == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(shape, seed, spread=0.0):
    g = _gen(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    if spread:  # rows of very different size
        x = x * torch.exp(spread * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))
    return x.to(BF16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _new(B, tokens, H, page, D, seed, fill=0xFF):
    """A cache whose every byte is `fill` (0xff: NaN codes and scales), and a table of scattered pages."""
    per = -(-tokens // page)
    pages = B * per + 2
    cache = fa.KVCache8.empty(pages, H, page, D)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.view(torch.uint8).fill_(fill)
    table = torch.randperm(pages, generator=_gen(seed), device="cuda")[:B * per].view(B, per).to(torch.int32)
    return cache, table


def _filled(B, lens, H, page, D, seed, spread=0.0):
    """A cache holding lens[b] tokens of each sequence (garbage elsewhere), its table and the values it
    holds: lists of k, v [H, lens[b], D]."""
    N = max(max(lens), 1)
    cache, table = _new(B, N, H, page, D, seed)
    k, v = _rand((B, H, N, D), seed + 1, spread), _rand((B, H, N, D), seed + 2, spread)
    fa.cache_write(cache, k, v, table, _ints([0] * B), _ints(lens))
    ks, vs = fa.cache_read(cache, table, _ints(lens), N)
    return cache, table, [ks[b, :, :n] for b, n in enumerate(lens)], [vs[b, :, :n] for b, n in enumerate(lens)]


def _close(out, lse, want, v, page, label="", few=True):
    o, l, a, size, spread = want
    n_keys = v.shape[1]
    dt = size * 2.0 ** -17 + spread * 2.0 ** -17.8 + 2.0 ** -21
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * dt[..., None] + n_keys / 32 * 2.0 ** -24) * a
    if n_keys:
        floor = 2.0 ** -24 * ref.weight(v.double(), page, few).sum(1)  # 2^-25, and the weight's factor of 2
        tol = tol + floor.repeat_interleave(out.shape[0] // v.shape[0], 0)[:, None]
    tol = tol * (1 + 2.0 ** -6) + 1e-30
    err = (out.double() - o).abs()
    assert bool((err <= tol).all()), (label, float((err / tol).max()))
    gone = torch.isneginf(l)
    assert torch.equal(torch.isneginf(lse), gone), label
    ltol = dt + 2.0 ** -21 * (1 + l.abs())
    lerr = (lse.double() - l).abs()
    assert bool((lerr <= ltol)[~gone].all()), (label, float((lerr / ltol)[~gone].max()))


def _check_all(q, cache, table, lens, ks, vs, causal, q_start=None, scale=None):
    out, lse = fa.fwd_cache(q, cache, table, _ints(lens), causal=causal, scale=scale,
                            q_start=None if q_start is None else _ints(q_start))
    torch.cuda.synchronize()
    assert fa.read_device_status() == 0
    s = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    for b, n in enumerate(lens):
        want = ref.attend(q[b], ks[b], vs[b], s, causal, None if q_start is None else q_start[b])
        _close(out[b], lse[b], want, vs[b], cache.k.shape[2], (b, n), q.shape[1] // ks[b].shape[0] * q.shape[2] <= 16)
    return out, lse


# ---- writing and reading back ----

@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("start,N", [(0, 1), (0, 300), (37, 128), (64, 131)])
def test_written_values_are_the_definition(D, page, start, N):
    """One call into an empty sequence (start rows of the first page hold nothing that counts)."""
    B, H = 3, 2
    counts = [N, N // 2, 0]
    cache, table = _new(B, start + N, H, page, D, 1)
    k = _rand((B, H, N, D), 2, 1.5)
    v = _rand((B, N, 3, H, D), 3, 1.5)[:, :, 1].transpose(1, 2)  # a slice of a projection
    if start % page:  # the first page's earlier tokens: zeros, which leave the scale to the new ones
        z = torch.zeros(B, H, start % page, D, dtype=BF16, device="cuda")
        fa.cache_write(cache, z, z, table, _ints([start // page * page] * B))
    fa.cache_write(cache, k, v, table, _ints([start] * B), _ints(counts))
    got = fa.cache_read(cache, table, _ints([start + n for n in counts]), N + 5, start=_ints([start] * B))
    for x, y in zip((k, v), got):
        for b, n in enumerate(counts):
            if n:
                want, _ = ref.quantised(x[b, :, :n], page, start)
                assert torch.equal(y[b, :, :n].double(), want), (b, float((y[b, :, :n].double() - want).abs().max()))
            assert not bool(y[b, :, n:].any())
    assert fa.read_device_status() == 0


def test_unaligned_inputs_give_the_same_codes():
    B, H, N, D, page = 2, 2, 77, 64, 32
    buf = _rand((B * H * N * (D + 1) + 1,), 4)
    x = buf[1:].view(B, H, N, D + 1)[..., :D]
    caches = []
    for k in (x, x.contiguous()):
        cache, table = _new(B, N, H, page, D, 5, fill=0)
        fa.cache_write(cache, k, k, table, _ints([0, 0]))
        caches.append(cache)
    assert torch.equal(caches[0].k.view(torch.uint8), caches[1].k.view(torch.uint8))
    assert torch.equal(caches[0].v_scale, caches[1].v_scale)


@pytest.mark.parametrize("sizes", [[1] * 40, [5, 1, 60, 3, 128, 7], [33, 33, 33, 33]])
def test_appending_in_pieces(sizes):
    """Scales end as if written at once; a value that was rounded again when its page's scale grew is
    off by half a step of e4m3 and half a subnormal step (2^-10 of the scale) more."""
    H, D, page = 2, 32, 64
    N = sum(sizes)
    x = _rand((1, H, N, D), 6, 2.0)  # sizes vary by e^2: scales grow often
    cache, table = _new(1, N, H, page, D, 7)
    held = 0
    for n in sizes:
        fa.cache_write(cache, x[:, :, held:held + n], x[:, :, held:held + n], table, _ints([held]))
        held += n
    got, _ = fa.cache_read(cache, table, _ints([N]), N)
    want, s = ref.quantised(x[0], page)
    ids = table[0].long()
    per_page = cache.k_scale[ids].double()  # [pages, H]
    assert torch.equal(per_page.T.repeat_interleave(page, 1)[:, :N], s)
    assert torch.equal(cache.k_scale[ids], cache.v_scale[ids])
    xd, err = x[0].double(), (got[0].double() - x[0].double()).abs()
    half = torch.maximum(xd.abs() * 2.0 ** -4, s[..., None] * 2.0 ** -10)
    assert bool((err <= half + s[..., None] * 2.0 ** -10).all())
    normal = want.abs() >= s[..., None] * 2.0 ** -5  # nothing below e4m3's normals on the way
    assert torch.equal(got[0].double()[normal], want[normal])


def test_rows_outside_the_call_are_left_alone():
    B, H, N, D, page = 2, 2, 50, 64, 64
    cache, table = _new(B, 200, H, page, D, 8, fill=0x31)
    before = cache.k.view(torch.uint8).clone()
    scale_before = cache.k_scale.clone()
    x = _rand((B, H, N, D), 9)
    fa.cache_write(cache, x, x, table, _ints([64, 128]), _ints([50, 20]))
    after = cache.k.view(torch.uint8)
    p0, p1 = int(table[0, 1]), int(table[1, 2])
    changed = (after != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert sorted(changed) == sorted([p0, p1])
    assert torch.equal(after[p0, :, 50:], before[p0, :, 50:]) and torch.equal(after[p1, :, 20:], before[p1, :, 20:])
    moved = (cache.k_scale.view(torch.int32) != scale_before.view(torch.int32)).any(1).nonzero().flatten().tolist()
    assert sorted(moved) == sorted([p0, p1])


def test_extreme_values():
    """Zeros, the least and the largest bf16 numbers, infinities and NaN."""
    H, D, page = 1, 32, 32
    x = torch.zeros(1, H, 5 * page, D, dtype=BF16, device="cuda")
    rows = x[0, 0].view(5, page, D)
    rows[1, 3, 7] = 9.2e-41       # the least subnormal: below half of the least step, 2^-10 * 2^-117
    rows[2, :, 0] = torch.finfo(BF16).max
    rows[2, :, 1] = -1.0
    rows[3, 0, 0], rows[3, 1, 1], rows[3, 2, 2], rows[3, 4, 5] = math.inf, -math.inf, math.nan, 3.0
    rows[4] = -448.0
    cache, table = _new(1, 5 * page, H, page, D, 10)
    fa.cache_write(cache, x, x, table, _ints([0]))
    got = fa.cache_read(cache, table, _ints([5 * page]), 5 * page)[0][0, 0].view(5, page, D)
    s = cache.k_scale[table[0].long()].flatten().tolist()
    assert s == [2.0 ** -117, 2.0 ** -117, 2.0 ** 119, 2.0 ** -7, 1.0]
    assert not bool(got[0].any()) and not bool(got[1].any())
    assert bool((got[2, :, 0].double() == 448.0 * 2.0 ** 119).all())   # saturates at the largest code
    assert not bool(got[2, :, 1].any())
    bad = torch.zeros(page, D, dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert torch.equal(got[3].isnan(), bad) and float(got[3, 4, 5]) == 3.0
    assert bool((got[4] == -448).all())


def test_offsets_past_32_bits():
    """Pages whose codes lie past 2^31 bytes, written, read and attended to."""
    H, D, page = 8, 128, 128
    pages = (1 << 31) // (H * D * page) + 40
    cache = fa.KVCache8.empty(pages, H, page, D)
    table = torch.arange(pages - 3, pages, dtype=torch.int32, device="cuda")[None]
    x, y = _rand((1, H, 300, D), 11), _rand((1, H, 300, D), 12)
    fa.cache_write(cache, x, y, table, _ints([0]))
    k, v = fa.cache_read(cache, table, _ints([300]), 300)
    assert torch.equal(k[0].double(), ref.quantised(x[0], page)[0])
    assert torch.equal(v[0].double(), ref.quantised(y[0], page)[0])
    _check_all(_rand((1, H, 2, D), 13), cache, table, [300], k, v, True)


# ---- attention ----

@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("g,Nq", [(1, 1), (4, 1), (2, 3), (8, 2), (3, 7)])
@pytest.mark.parametrize("causal", [False, True])
def test_few_rows(D, page, g, Nq, causal):
    lens = [1 if Nq == 1 else Nq, 31 + Nq, 128, 129, 777]
    cache, table, ks, vs = _filled(len(lens), lens, 2, page, D, 20)
    _check_all(_rand((len(lens), 2 * g, Nq, D), 21), cache, table, lens, ks, vs, causal)


@pytest.mark.parametrize("D,page,Hk,g", [(128, 128, 2, 1), (64, 64, 1, 4), (32, 32, 2, 2)])
@pytest.mark.parametrize("Nq", [16, 17, 32, 33])
@pytest.mark.parametrize("causal", [False, True])
def test_around_the_row_counts_that_choose_a_kernel(D, page, Hk, g, Nq, causal):
    """16 and 17 rows of a key head, 128 and 129 and 132: few rows, pairs of key tiles, two row tiles."""
    lens = [Nq, 140, 2300]
    cache, table, ks, vs = _filled(3, lens, Hk, page, D, 25)
    _check_all(_rand((3, Hk * g, Nq, D), 26), cache, table, lens, ks, vs, causal)


@pytest.mark.parametrize("Nq", [1, 9, 40])
def test_many_sequences(Nq):
    """More sequences than lanes of a warp, of all lengths, some empty."""
    B = 75
    lens = [(b * 37) % 301 for b in range(B)]
    cache, table, ks, vs = _filled(B, lens, 1, 32, 32, 35)
    _check_all(_rand((B, 2, Nq, 32), 36), cache, table, lens, ks, vs, True)


@pytest.mark.parametrize("L", [1, 2, 32, 33, 127, 128, 255, 256, 1000, 20011])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_lengths_of_one_sequence(L, D):
    cache, table, ks, vs = _filled(1, [L], 3, 64, D, 30)
    _check_all(_rand((1, 6, 1, D), 31), cache, table, [L], ks, vs, False)


@pytest.mark.parametrize("D,page,Hk,g", [(128, 128, 2, 1), (64, 32, 2, 4), (32, 64, 1, 2), (128, 64, 1, 3)])
@pytest.mark.parametrize("Nq", [17, 64, 130, 513])
@pytest.mark.parametrize("causal", [False, True])
def test_chunks(D, page, Hk, g, Nq, causal):
    lens = [Nq, Nq + 301, 1500]
    cache, table, ks, vs = _filled(3, lens, Hk, page, D, 40)
    _check_all(_rand((3, Hk * g, Nq, D), 41), cache, table, lens, ks, vs, causal)


@pytest.mark.parametrize("Nq", [1, 5, 200])
def test_empty_sequences_and_rows_before_the_first_key(Nq):
    """Length 0; fewer keys than rows (the first rows see none); rows placed by q_start."""
    lens = [0, 3, 0, 70]
    cache, table, ks, vs = _filled(4, lens, 2, 32, 64, 50)
    q = _rand((4, 4, Nq, 64), 51)
    out, lse = _check_all(q, cache, table, lens, ks, vs, True)
    assert not bool(out[0].any()) and bool(torch.isneginf(lse[0]).all())
    if Nq == 5:
        assert not bool(out[1, :, :2].any()) and bool(torch.isneginf(lse[1, :, :2]).all())
    _check_all(q, cache, table, lens, ks, vs, False)
    _check_all(q, cache, table, lens, ks, vs, True, q_start=[0, -2, 5, 30])
    _check_all(q, cache, table, lens, ks, vs, True, q_start=[-2 ** 31, -Nq, 2 ** 31 - 1, 2 ** 31 - 1])


@pytest.mark.parametrize("Nq", [1, 300])
def test_what_lies_past_the_length_is_not_read(Nq):
    """NaN codes and scales in every other page and row, and table entries outside the cache."""
    lens = [200, 65]
    cache, table, ks, vs = _filled(2, lens, 2, 32, 64, 60)
    table = torch.cat([table, torch.full((2, 4), -7, dtype=torch.int32, device="cuda")], 1).contiguous()
    table[1, 3:] = 2 ** 31 - 1
    _check_all(_rand((2, 4, Nq, 64), 61), cache, table, lens, ks, vs, True)


@pytest.mark.parametrize("Nq", [1, 6, 300])
def test_scales_that_differ_between_pages(Nq):
    """Tokens whose sizes vary over several powers of ten, so neighbouring pages have unlike scales."""
    lens = [900, 333]
    cache, table, ks, vs = _filled(2, lens, 2, 32, 64, 70, spread=2.0)
    _check_all(_rand((2, 4, Nq, 64), 71), cache, table, lens, ks, vs, True, scale=0.02)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("Nq", [1, 300])
def test_scales_of_the_scores(scale, Nq):
    """Uniform, negative and very sharp softmax."""
    cache, table, ks, vs = _filled(2, [500, 131], 1, 64, 32, 80)
    _check_all(_rand((2, 2, Nq, 32), 81), cache, table, [500, 131], ks, vs, False, scale=scale)


@pytest.mark.parametrize("rows", [1, 20, 140])
def test_a_sink_and_a_long_tail(rows):
    """One key far above 40,000 others that together weigh as much as it does: probabilities of 2^-16
    of the largest still count."""
    L, D = 40000, 64
    cache, table = _new(1, L, 1, 128, D, 90)
    k, v = torch.zeros(1, 1, L, D, dtype=BF16, device="cuda"), _rand((1, 1, L, D), 91)
    k[:, :, 5, 0] = 1.0
    v[..., 1] = 1.0
    fa.cache_write(cache, k, v, table, _ints([0]))
    ks, vs = fa.cache_read(cache, table, _ints([L]), L)
    q = torch.zeros(1, 1, rows, D, dtype=BF16, device="cuda")
    q[..., 0] = 10.625  # ln 40000 = 10.6
    out, _ = _check_all(q, cache, table, [L], ks, vs, False, scale=1.0)
    assert float((out[..., 1] - 1).abs().max()) <= 2.0 ** -8


@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_huge_scores_of_few_rows(sign):
    """Equal scores of +-1.1e31 on every key: a uniform softmax, with LSE the score itself.  (Equal
    keys give equal scores, so every p is a power of two: O is the mean but for fp32 sums and the last
    rounding, 2^-8 |O| + 2^-20 of the mean of |v|.  LSE: 2^-17.8 from q, less than 2^-18 from the rest.)"""
    L, D = 700, 64
    cache, table = _new(1, L, 1, 64, D, 95)
    k, v = torch.full((1, 1, L, D), sign * 1.2e15, dtype=BF16, device="cuda"), _rand((1, 1, L, D), 96)
    fa.cache_write(cache, k, v, table, _ints([0]))
    ks, vs = fa.cache_read(cache, table, _ints([L]), L)
    q = torch.full((1, 1, 1, D), 1.2e15, dtype=BF16, device="cuda")
    out, lse = fa.fwd_cache(q, cache, table, _ints([L]), scale=0.125)
    score = float((q[0, 0, 0].double() * ks[0, 0, 0].double()).sum()) * 0.125
    assert 1e31 < abs(score) < 1.3e31
    mean, size = vs[0, 0].double().mean(0), vs[0, 0].double().abs().mean(0)
    assert bool(((out[0, 0].double() - mean).abs() <= 2.0 ** -8 * mean.abs() + 2.0 ** -20 * size).all())
    assert bool(((lse.double() - score).abs() <= 2.0 ** -17 * abs(score)).all())


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("rows", [1, 20, 140])
def test_large_scores(rows, sign):
    """Scores around +-2^15."""
    L, D = 700, 64
    cache, table = _new(1, L, 1, 64, D, 97)
    k, v = _rand((1, 1, L, D), 98), _rand((1, 1, L, D), 99)
    k[..., 0] = sign * 512.0
    fa.cache_write(cache, k, v, table, _ints([0]))
    ks, vs = fa.cache_read(cache, table, _ints([L]), L)
    q = _rand((1, 1, rows, D), 100)
    q[..., 0] = 512.0
    _check_all(q, cache, table, [L], ks, vs, False, scale=0.125)


@pytest.mark.parametrize("g", [4, 24, 150])
def test_rows_that_are_not_finite_stay_apart(g):
    """A NaN or infinite query row gives NaN and leaves the other rows alone; so does a NaN key for the
    rows that do not see it."""
    cache, table, ks, vs = _filled(1, [300], 1, 64, 64, 100)
    q = _rand((1, g, 1, 64), 101)
    want, _ = fa.fwd_cache(q, cache, table, _ints([300]))
    q[0, 1, 0, 3], q[0, 2, 0, 60] = math.nan, math.inf
    out, lse = fa.fwd_cache(q, cache, table, _ints([300]))
    assert bool(out[0, 1:3].isnan().all()) and bool(lse[0, 1:3].isnan().all())
    assert torch.equal(out[0, 0], want[0, 0]) and torch.equal(out[0, 3], want[0, 3])
    k = torch.full((1, 1, 1, 64), math.nan, dtype=BF16, device="cuda")
    fa.cache_write(cache, k, _rand((1, 1, 1, 64), 102), table, _ints([299]))
    q = _rand((1, g, 3, 64), 103)
    out, lse = fa.fwd_cache(q, cache, table, _ints([300]), causal=True)  # rows 0, 1 do not see key 299
    assert bool(out[0, :, :2].isfinite().all()) and bool(out[0, :, 2].isnan().all()) and bool(lse[0, :, 2].isnan().all())


@pytest.mark.parametrize("Nq", [1, 200])
def test_shared_pages(Nq):
    """Two sequences that share their first pages (a common prompt)."""
    cache, table, ks, vs = _filled(1, [300], 2, 64, 64, 110)
    both = torch.stack([table[0], table[0]])
    q = _rand((2, 2, Nq, 64), 111)
    _check_all(q, cache, both, [300, 190], [ks[0], ks[0][:, :190]], [vs[0], vs[0][:, :190]], True)


@pytest.mark.parametrize("Nq", [1, 9, 300])
def test_repeatable_on_streams_and_in_graphs(Nq):
    lens = [3000, 1, 0, 1777]
    cache, table, ks, vs = _filled(4, lens, 2, 64, 128, 120)
    q, n = _rand((4, 4, Nq, 128), 121), _ints(lens)
    want = fa.fwd_cache(q, cache, table, n, causal=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, s.cuda_stream):
        got = fa.fwd_cache(q, cache, table, n, causal=True, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two captured graphs, replayed in turn, then with other lengths
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, fa.fwd_cache(q, cache, table, n, causal=True)))
        graphs[-1] = (g, graphs[-1][1])
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    n.copy_(_ints([5, 900, 64, 0]))
    want = fa.fwd_cache(q, cache, table, n, causal=True)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.nan_to_num(0), b.nan_to_num(0)) for a, b in zip(graphs[0][1], want))
    assert fa.read_device_status() == 0


def test_chunk_by_chunk_against_the_whole():
    """Rotary positions, the cache and the attention together, as a model that generates frame by frame
    (then token by token) uses them, against the definition on what the cache holds."""
    B, Hq, Hk, D, page = 2, 4, 2, 64, 32
    grid = torch.cartesian_prod(torch.arange(5), torch.arange(6), torch.arange(7)).to(torch.int32).cuda()
    axes = fa.RopeAxes((16, 24, 24), theta=256.0)
    sizes = [42 * 2, 42, 1, 1, 1, 42]
    N = sum(sizes)
    x = _rand((B, N, Hq + 2 * Hk, D), 130)
    cache, table = _new(B, N, Hk, page, D, 131)
    held = 0
    for n in sizes:
        part = x[:, held:held + n]
        q, k, v = (part[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        q, k = fa.rope(q, k, grid[held:held + n], axes)
        fa.cache_write(cache, k, v, table, _ints([held] * B))
        held += n
        out, lse = fa.fwd_cache(q, cache, table, _ints([held] * B), causal=True)
        ks, vs = fa.cache_read(cache, table, _ints([held] * B), held)
        for b in range(B):
            _close(out[b], lse[b], ref.attend(q[b], ks[b], vs[b], D ** -0.5, True), vs[b], page, held,
                   Hq // Hk * n <= 16)
    # what the cache holds is what was written, to e4m3's precision
    kx = ref.rope(x[:, :, Hq:Hq + Hk].transpose(1, 2), grid[:N], axes.dims, 256.0)
    err = (ks.double() - kx).abs().amax() / kx.abs().amax()
    assert float(err) <= 2.0 ** -4 + 2.0 ** -8
    assert fa.read_device_status() == 0


# ---- numbers in device memory that are out of range ----

def test_index_errors_are_recorded_and_write_nothing():
    B, H, D, page = 2, 1, 32, 32
    cache, table = _new(B, 64, H, page, D, 140, fill=0)
    x = _rand((B, H, 8, D), 141)
    for tab, start, count in ((_ints([[99, 0], [-1, 0]]), [0, 0], [8, 8]), (table, [-1, 64], [0, 0]),
                              (table, [64, 2 ** 31 - 1], [8, 8]), (table, [0, 0], [-1, -2 ** 31])):
        fa.cache_write(cache, x, x, tab.contiguous(), _ints(start), _ints(count))
        assert fa.read_device_status() == FA_ERR_INDEX
        assert not bool(cache.k.view(torch.uint8).any())
    fa.cache_write(cache, x, x, table, _ints([60, 0]), _ints([8, 0]))  # four of eight tokens have a place
    assert fa.read_device_status() == FA_ERR_INDEX
    k, _ = fa.cache_read(cache, table, _ints([64, 0]), 4, start=_ints([60, 0]))
    assert torch.equal(k[0].double(), ref.quantised(x[0, :, :4], page, 60)[0])
    assert fa.read_device_status() == 0
    fa.cache_read(cache, table, _ints([65, -1]), 4)
    assert fa.read_device_status() == FA_ERR_INDEX
    for Nq in (1, 200):
        q = _rand((B, H, Nq, D), 142)
        fa.fwd_cache(q, cache, table, _ints([1000, 5]))
        assert fa.read_device_status() == FA_ERR_INDEX
        fa.fwd_cache(q, cache, _ints([[0, 500], [1, -9]]), _ints([40, 40]))
        assert fa.read_device_status() == FA_ERR_INDEX
        fa.fwd_cache(q, cache, table, _ints([40, 40]))
        assert fa.read_device_status() == 0


@pytest.mark.parametrize("Nq", [1, 40, 300])
def test_withheld_tile_times_out_and_the_context_survives(monkeypatch, Nq):
    """CTA 0 withholds its second tile of keys: its waits run out, the call ends and the next is right."""
    cache, table, ks, vs = _filled(1, [5000], 1, 64, 64, 150)
    q = _rand((1, 1, Nq, 64), 151)
    wide = table.repeat(1, 400)  # more tiles than CTAs, so that CTA 0 has a second one
    monkeypatch.setenv("FA_FAULT_INJECT", "stall")
    monkeypatch.setenv("FA_WAIT_TIMEOUT_MS", "100")
    fa.fwd_cache(q, cache, wide, _ints([5000 * 300]))
    torch.cuda.synchronize()
    assert fa.read_device_status() == FA_ERR_TIMEOUT
    monkeypatch.delenv("FA_FAULT_INJECT")
    monkeypatch.delenv("FA_WAIT_TIMEOUT_MS")
    _check_all(q, cache, table, [5000], ks, vs, False)


CHILD_CAPTURE = r"""
import sys, torch
sys.path.insert(0, ROOT)
import unet_fa_fwd_gb300 as fa
torch.cuda.set_device(0)
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(2, 130, 8, 64, generator=g, device="cuda").bfloat16()
q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, 4), (4, 6), (6, 8)))
pos = torch.arange(130, dtype=torch.int32, device="cuda")[:, None].expand(130, 3).contiguous()
axes = fa.RopeAxes((16, 24, 24))
cache = fa.KVCache8.empty(20, 2, 32, 64)
table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
zero, n = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.full((2,), 130, dtype=torch.int32, device="cuda")

def step():
    a, b = fa.rope(q, k, pos, axes)
    fa.cache_write(cache, b, v, table, zero)
    out = [fa.fwd_cache(a, cache, table, n, causal=True)]
    out.append(fa.fwd_cache(a[:, :, 129:].contiguous(), cache, table, n))
    return out + [fa.cache_read(cache, table, n, 130)]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):  # the process's first calls
    got = step()
graph.replay()
torch.cuda.synchronize()
want = step()
torch.cuda.synchronize()
assert fa.read_device_status() == 0 and fa.debug_report() == [0] * 8
for a, b in zip(got, want):
    assert all(torch.equal(x, y) for x, y in zip(a, b))
print("same")
"""


@pytest.mark.parametrize("debug", ["0", "1"])
def test_first_calls_inside_a_capture(debug):
    """A whole step captured before anything else ran, replayed, against the same step run eagerly; in the
    release build and in the debug build, whose checks must find nothing."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", CHILD_CAPTURE.replace("ROOT", repr(root))], capture_output=True,
                         text=True, timeout=300, env=dict(os.environ, FA_DEBUG=debug))
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stdout + out.stderr


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own workspace."""
    lens = [9000, 777]
    cache, table, ks, vs = _filled(2, lens, 4, 64, 64, 155)
    n = _ints(lens)
    qs = [_rand((2, 8, 1, 64), 156), _rand((2, 4, 50, 64), 157)]
    want = [fa.fwd_cache(q, cache, table, n, causal=True) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (q, s) in enumerate(zip(qs, streams)):
            got[i].append(fa.fwd_cache(q, cache, table, n, causal=True, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_refusals():
    cache, table, _, _ = _filled(2, [40, 40], 2, 32, 64, 160)
    q, n = _rand((2, 4, 1, 64), 161), _ints([40, 40])
    with pytest.raises(RuntimeError, match="INVALID_ARGUMENT"):
        fa.fwd_cache(q[:, :3].contiguous(), cache, table, n)          # 3 query heads on 2 key heads
    with pytest.raises(ValueError, match="heads of 64"):
        fa.fwd_cache(_rand((2, 4, 1, 32), 1), cache, table, n)
    with pytest.raises(ValueError, match="contiguous"):
        fa.fwd_cache(_rand((2, 1, 4, 64), 1).transpose(1, 2).expand(2, 4, 2, 64), cache, table, n)
    with pytest.raises(TypeError, match="int32"):
        fa.fwd_cache(q, cache, table.long(), n)
    with pytest.raises(ValueError, match="lens must have shape"):
        fa.fwd_cache(q, cache, table, n[:1])
    with pytest.raises(ValueError, match="must be"):
        fa.fwd_cache(q, cache, table, n.cpu())
    with pytest.raises(TypeError, match="bfloat16"):
        fa.cache_write(cache, q[:, :2].float(), q[:, :2], table, n)
    with pytest.raises(ValueError, match="heads of"):
        fa.cache_write(cache, q, q, table, n)
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        c = fa.KVCache8.empty(4, 2, 16, 64)
        fa.cache_read(c, table, n, 3)
    with pytest.raises(RuntimeError, match="INVALID_ARGUMENT"):
        need = fa.cache_workspace_bytes(2, 4, 2, 1, 64, 400, 32)
        wide = table.repeat(1, 200)
        fa.fa_fwd_cache(q, cache, wide, n, torch.empty_like(q), torch.empty(2, 4, 1, device="cuda"),
                        torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="k_scale"):
        fa.KVCache8(cache.k, cache.v, cache.k_scale[:1], cache.v_scale)
