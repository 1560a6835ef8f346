"""Which layouts of outputs and inputs fa_rope takes, without a GPU: an output may be its input, else it
shares no element with the inputs or the other output, and no element is written twice.  Strides of
axes of size 1 are not used.  The launch hook ends an accepted call before any CUDA call."""
import ctypes
import itertools
import random

import pytest

import unet_fa_fwd_gb300 as fa
from unet_fa_fwd_gb300 import _build
from unet_fa_fwd_gb300.binding import FA_ERR_CUDA, FaRopeAxes, FaTensor

BASE, POS = 1 << 44, 1 << 50


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


@pytest.fixture(autouse=True)
def _hook(monkeypatch):
    monkeypatch.setenv("FA_FAULT_INJECT", "launch")


def _call(lib, q, qo, Hq, k, ko, Hk, B, N, D):
    """Tensors as (offset in bf16 elements, strides of B, H, N); True if taken."""
    axes = FaRopeAxes(count=1)
    axes.dims[0], axes.theta[0], axes.scale[0] = D, 1e4, 1.0
    t = [FaTensor(BASE + 2 * x[0], *x[1]) if x else None for x in (q, qo, k, ko)]
    ref = [ctypes.byref(x) if x else None for x in t]
    rc = lib.fa_rope(ctypes.byref(axes), POS, 0, ref[0], ref[1], Hq, ref[2], ref[3], Hk, B, N, D, 0, 0, 0, None)
    assert rc in (1, FA_ERR_CUDA)
    return rc == FA_ERR_CUDA


def test_slices_of_one_buffer_in_place(lib):
    B, Hq, Hk, N, D = 2, 4, 2, 10, 64
    H = Hq + 2 * Hk
    layouts = {
        "token-major": ((H * N * D, D, H * D), Hq * D),                   # [B, N, H, D]
        "head-major": ((H * N * D, N * D, D), Hq * N * D),                # [B, H, N, D]
        "sequence first": ((H * D, D, B * H * D), Hq * D),                # [N, B, H, D]
        "heads first": ((N * D, B * N * D, D), Hq * B * N * D),           # [H, B, N, D]
    }
    for name, (st, at) in layouts.items():
        q, k = (0, st), (at, st)
        assert _call(lib, q, q, Hq, k, k, Hk, B, N, D), name
        assert not _call(lib, q, q, Hq, (at - D, st), (at - D, st), Hk, B, N, D), name  # q's last row, or head
        # rotated into the next layer's slices of the same buffer
        assert _call(lib, k, (at + (at // Hq) * Hk, st), Hk, None, None, 0, B, N, D), name
    # q, k and v side by side in each head: [B, N, H, 3, D]
    st = (N * 4 * 3 * D, 3 * D, 4 * 3 * D)
    assert _call(lib, (0, st), (0, st), 4, (D, st), (D, st), 4, B, N, D)
    assert not _call(lib, (0, st), (0, st), 4, (D // 2, st), (D // 2, st), 4, B, N, D)


def test_strides_of_axes_of_size_one_are_not_used(lib):
    N, D = 7, 64
    assert _call(lib, (0, (5, 3 * N * D, D)), (0, (11, 3 * N * D, D)), 2, None, None, 0, 1, N, D)
    assert _call(lib, (0, (5, 13, D)), (0, (11, 17, D)), 1, None, None, 0, 1, N, D)
    # one token of each of 3 sequences, q and k in a packed buffer, as different views of it give the strides
    assert _call(lib, (0, (6 * D, D, 6 * D)), (0, (6 * D, D, 1)), 4, (4 * D, (6 * D, D, 0)), (4 * D, (6 * D, D, 9)), 2,
                 3, 1, D)


def _elements(x, B, H, N, D):
    return [x[0] + b * x[1][0] + h * x[1][1] + n * x[1][2] for b, h, n in itertools.product(range(B), range(H), range(N))]


def _definition(q, qo, Hq, k, ko, Hk, B, N, D):
    def meet(a, b):
        return any(abs(x - y) < D for x in a for y in b)

    ins = [_elements(q, B, Hq, N, D), _elements(k, B, Hk, N, D)]
    outs = [_elements(qo, B, Hq, N, D), _elements(ko, B, Hk, N, D)]
    for i in range(2):
        if any(abs(x - y) < D for x, y in itertools.combinations(outs[i], 2)):
            return False
        for j in range(2):
            if not (i == j and outs[i] == ins[j]) and meet(outs[i], ins[j]):
                return False
    return not meet(outs[0], outs[1])


def test_against_the_elements_themselves(lib):
    """Drawn layouts: packed ones in every order of the axes, some bent; all offsets are looked at."""
    r = random.Random(5)
    taken = 0
    for _ in range(6000):
        B, N, Hq, Hk, D = r.randint(1, 3), r.randint(1, 4), r.randint(1, 3), r.randint(1, 3), 32

        def packed(H, extra):
            order, st, size = r.sample(range(3), 3), [0, 0, 0], D * r.choice((1, 1, 2, 3))
            for a in order:
                st[a] = size
                size *= (B, H + extra, N)[a] + r.choice((0, 0, 1))
            return tuple(st)

        st = packed(Hq + Hk, r.randint(0, 2))
        step = st[1] * Hq if r.random() < 0.6 else r.choice((D, D * N, D // 2, st[0], st[2], st[1]))
        q, k = (0, st), (step, st)
        bend = lambda x: (x[0], tuple(s + r.choice((0, 0, 0, D, -D if s > D else 0)) for s in x[1]))  # noqa: E731
        pick = r.random()
        if pick < 0.4:
            qo, ko = q, k
        elif pick < 0.7:
            at = r.choice((2 * step, D * r.randint(0, 60)))
            qo, ko = (at, st), (at + step, st)
        else:
            qo, ko = bend(q), bend(k)
        if r.random() < 0.2:
            q = (q[0], tuple(0 if r.random() < 0.3 else s for s in q[1]))
        got, want = _call(lib, q, qo, Hq, k, ko, Hk, B, N, D), _definition(q, qo, Hq, k, ko, Hk, B, N, D)
        taken += want
        assert got == want, (q, qo, Hq, k, ko, Hk, B, N)
    assert 600 < taken < 5400
