"""Rotary positions and the paged e4m3 cache without a GPU: index arithmetic
(fa_cache_geom.h, compiled with the host C++ compiler) and refusals, all of them
before any CUDA call."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import unet_fa_fwd_gb300 as fa
from unet_fa_fwd_gb300 import _build
from unet_fa_fwd_gb300.binding import FaCache, FaRopeAxes, FaTensor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "unet_fa_fwd_gb300", "csrc")
GB = 1 << 30
FAR = [i << 44 for i in range(1, 20)]  # addresses of buffers that do not meet


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


def test_index_arithmetic_matches_definition(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "cache_geom_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe),
                    os.path.join(HERE, "cache_geom_check.cpp")], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr


def test_status_name(lib):
    assert fa.status_string(6) == "FA_ERR_INDEX"


# ---- fa_rope ----

def _rope(lib, axes=((16, 56, 56), 10000.0, 1.0), pos=FAR[0], pos_b=0, q=None, qo=None, Hq=4, k=None, ko=None, Hk=2,
          B=2, N=10, D=128, dtype=0, pairing=0, no_k=False):
    a = None
    if axes is not None:
        dims, theta, scale = axes
        a = FaRopeAxes(count=len(dims))
        n = min(len(dims), 4)
        a.dims[:n], a.theta[:n], a.scale[:n] = dims[:n], (theta,) * n, (scale,) * n
        a = ctypes.byref(a)
    t = {}
    for name, given, at, H in (("q", q, 1, Hq), ("qo", qo, 2, Hq), ("k", k, 3, Hk), ("ko", ko, 4, Hk)):
        base = (FAR[at], H * N * D, N * D, D)
        t[name] = FaTensor(*(base if given is None else given))
    ref = {n: ctypes.byref(v) for n, v in t.items()}
    if no_k:
        ref["k"] = ref["ko"] = None
    return lib.fa_rope(a, pos, pos_b, ref["q"], ref["qo"], Hq, ref["k"], ref["ko"], Hk, B, N, D, dtype, pairing, 0,
                       None)


S = (4 * 10 * 128, 10 * 128, 128)  # contiguous strides of q
PACKED = (10 * 8 * 128, 128, 8 * 128)  # a token-major buffer of 8 heads


@pytest.mark.parametrize("kw,code", [
    (dict(axes=None), 1), (dict(pos=None), 1), (dict(q=(None, *S)), 1), (dict(B=0), 1), (dict(N=0), 1),
    (dict(Hq=0), 1), (dict(Hk=0), 1), (dict(D=48), 2), (dict(dtype=3), 2), (dict(pairing=2), 1),
    (dict(axes=((16, 56), 1e4, 1.0)), 1),                   # sums to 72
    (dict(axes=((15, 57, 56), 1e4, 1.0)), 1),               # odd
    (dict(axes=((0, 72, 56), 1e4, 1.0)), 1),
    (dict(axes=((32,) * 5, 1e4, 1.0)), 1),                  # five axes
    (dict(axes=((16, 56, 56), 0.0, 1.0)), 1), (dict(axes=((16, 56, 56), math.nan, 1.0)), 1),
    (dict(axes=((16, 56, 56), 1e4, math.inf)), 1),
    (dict(pos=FAR[0] + 2), 1), (dict(pos_b=-1), 1),
    (dict(q=(FAR[1], -S[0], S[1], S[2])), 1),               # negative stride
    (dict(q=(FAR[1] + 1, *S)), 1),                          # half an element
    (dict(qo=(FAR[2], S[0], 0, S[2])), 1),                  # an output written twice
    (dict(qo=(FAR[2], S[0], S[1], 64)), 1),
    (dict(qo=(FAR[1] + 256, *S)), 1),                       # the output one row behind its input
    (dict(ko=(FAR[2], *S)), 1),                             # two outputs in one place
    (dict(qo=(FAR[0] - 64, *S)), 1),                        # positions inside the output
    (dict(q=(FAR[1], *PACKED), k=(FAR[1] + 4 * 256, *PACKED), qo=(FAR[1] + 256, *PACKED)), 1),
    (dict(q=(FAR[1], 1 << 61, 1, 1)), 1),                   # offsets past 64 bits
])
def test_rope_refusals(lib, kw, code):
    assert _rope(lib, **kw) == code


@pytest.mark.parametrize("kw", [
    {}, dict(no_k=True), dict(qo=(FAR[1], *S)),                                # in place
    dict(q=(FAR[1], *PACKED), k=(FAR[1] + 4 * 256, *PACKED)),                  # slices of one projection
    dict(qo=(FAR[2], *PACKED), ko=(FAR[2] + 4 * 256, *PACKED)),
    dict(q=(FAR[1], *PACKED), k=(FAR[1] + 1024, *PACKED), qo=(FAR[1], *PACKED), ko=(FAR[1] + 1024, *PACKED)),
    dict(q=(FAR[1], 0, 0, 0)),                                                 # broadcast input
    dict(N=1, qo=(FAR[2], 4 * 128, 128, 0)), dict(dtype=2), dict(pairing=1), dict(q=(FAR[1] + 2, *S)),
])
def test_rope_accepts(lib, kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _rope(lib, **kw) == 3   # the first CUDA call


# ---- the cache ----

def _cache(**kw):
    a = dict(k=FAR[5], v=FAR[6], k_scale=FAR[7], v_scale=FAR[8], num_pages=10, H=2, page_tokens=64, D=64)
    a.update(kw)
    return FaCache(*(a[n] for n in ("k", "v", "k_scale", "v_scale", "num_pages", "H", "page_tokens", "D")))


BAD_CACHES = [
    (dict(k=None), 1), (dict(v_scale=None), 1), (dict(k=FAR[5] + 8), 1), (dict(k_scale=FAR[7] + 2), 1),
    (dict(num_pages=0), 1), (dict(H=0), 1), (dict(D=48), 2), (dict(page_tokens=16), 2), (dict(page_tokens=256), 2),
    (dict(num_pages=1 << 30, H=8), 1), (dict(v=FAR[5] + 64), 1), (dict(v_scale=FAR[7] + 8), 1),
    (dict(k_scale=FAR[6] + 64), 1),
]
CS = (2 * 9 * 64, 9 * 64, 64)


def _write(lib, cache=None, k=None, v=None, table=FAR[0], width=3, start=FAR[1], count=FAR[2], B=2, N=9):
    c = _cache(**(cache or {}))
    k, v = (FaTensor(*(t or (FAR[at], *CS))) for t, at in ((k, 3), (v, 4)))
    return lib.fa_cache_write(ctypes.byref(c), ctypes.byref(k), ctypes.byref(v), table, width, start, count, B, N, None)


def _read(lib, cache=None, table=FAR[0], width=3, lens=FAR[1], first=FAR[2], k=FAR[3], v=FAR[4], B=2, N=9):
    c = _cache(**(cache or {}))
    return lib.fa_cache_read(ctypes.byref(c), table, width, lens, first, k, v, B, N, None)


def _attend(lib, cache=None, q=FAR[9], table=FAR[0], width=3, lens=FAR[1], q_start=FAR[2], out=FAR[3], lse=FAR[4],
            B=2, Hq=4, Nq=5, scale=0.125, ws=FAR[10], ws_bytes=GB):
    c = _cache(**(cache or {}))
    return lib.fa_fwd_cache(q, ctypes.byref(c), table, width, lens, q_start, 1, out, lse, B, Hq, Nq,
                            ctypes.c_float(scale), ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_write, _read, _attend])
@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, call, kw, code):
    assert call(lib, cache=kw) == code


@pytest.mark.parametrize("call,kw", [
    (_write, dict(table=None)), (_write, dict(table=FAR[0] + 1)), (_write, dict(width=0)), (_write, dict(B=0)),
    (_write, dict(N=0)), (_write, dict(start=None)), (_write, dict(count=FAR[2] + 2)),
    (_write, dict(k=(None, *CS))), (_write, dict(k=(FAR[3] + 1, *CS))), (_write, dict(v=(FAR[4], -1, 64, 64))),
    (_write, dict(k=(FAR[5] + 32, *CS))),                       # inside the cache
    (_write, dict(start=FAR[7])), (_write, dict(table=FAR[5])),
    (_write, dict(width=(1 << 25) - 1, N=1 << 12)),             # positions past 32 bits
    (_write, dict(B=1 << 30)),
    (_read, dict(lens=None)), (_read, dict(k=None)), (_read, dict(v=FAR[4] + 8)), (_read, dict(N=0)),
    (_read, dict(k=FAR[4] + 64)), (_read, dict(k=FAR[5])), (_read, dict(v=FAR[0] - 16)), (_read, dict(B=1 << 30)),
    (_attend, dict(q=None)), (_attend, dict(out=None)), (_attend, dict(lse=None)), (_attend, dict(lens=None)),
    (_attend, dict(q=FAR[9] + 8)), (_attend, dict(out=FAR[9])), (_attend, dict(lse=FAR[3] + 16)),
    (_attend, dict(out=FAR[5])), (_attend, dict(lse=FAR[0])), (_attend, dict(q_start=FAR[2] + 1)),
    (_attend, dict(Hq=5)), (_attend, dict(Hq=0)), (_attend, dict(Nq=0)), (_attend, dict(B=0)),
    (_attend, dict(scale=math.nan)), (_attend, dict(scale=math.inf)),
    (_attend, dict(B=1 << 16, Nq=1 << 14)),                     # 2^32 rows
    (_attend, dict(B=1 << 30, Hq=1 << 30, Nq=1 << 30)),         # sizes whose products pass 64 bits
    (_write, dict(cache=dict(num_pages=1, H=1 << 29), B=1 << 30, N=1922, k=(FAR[3], 0, 0, 0), v=(FAR[4], 0, 0, 0))),
    (_read, dict(cache=dict(num_pages=1, H=1 << 28), k=FAR[11], v=FAR[12], B=1 << 30, N=1 << 16)),
])
def test_bad_arguments_are_refused(lib, call, kw):
    assert call(lib, **kw) == 1


@pytest.mark.parametrize("call,kw", [
    (_write, {}), (_write, dict(count=None)), (_write, dict(k=(FAR[3], 0, 0, 0))), (_write, dict(k=(FAR[3] + 2, *CS))),
    (_read, {}), (_read, dict(first=None)), (_attend, {}), (_attend, dict(q_start=None)), (_attend, dict(scale=0.0)),
    (_attend, dict(scale=-1.0)),
])
def test_valid_calls_reach_the_device(lib, call, kw, monkeypatch):
    monkeypatch.setenv("FA_FAULT_INJECT", "launch")
    assert call(lib, **kw) == 3


def test_workspace_bytes(lib):
    size = lib.fa_cache_workspace_bytes
    # sequences of at most one tile need none; past that, room for 2 x 1024 stretches of 4 rows at most
    assert size(64, 32, 8, 1, 128, 2, 64) == 0
    assert size(64, 32, 8, 1, 128, 128, 64) == 2 * 1024 * 4 * (128 + 2) * 4 + 1024 * 16
    for bad in ((0, 1, 1, 1, 64, 9, 64), (1, 3, 2, 1, 64, 9, 64), (1, 1, 1, 1, 48, 9, 64),
                (1 << 30, 1 << 30, 1 << 30, 1 << 30, 64, 9, 64), (1, 1, 1, 1, 64, 1 << 30, 64)):
        assert size(*bad) == 0


# ---- the Python entry points ----

def test_python_checks():
    with pytest.raises(ValueError, match="axes"):
        fa.RopeAxes((8,) * 5)
    with pytest.raises(ValueError, match="theta"):
        fa.RopeAxes((16, 16), theta=(1.0,))
    axes = fa.RopeAxes((8, 12, 12), theta=(10.0, 20.0, 30.0))
    assert axes.scale == (1.0, 1.0, 1.0)
    x, pos = torch.zeros(1, 2, 5, 32, dtype=torch.bfloat16), torch.zeros(5, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.rope(x, x, pos, axes)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_rope(x, None, pos, axes, x, None)
    with pytest.raises(TypeError, match="q_out"):
        fa.fa_rope(x, None, pos, axes, None, None)
    with pytest.raises(TypeError, match="out"):
        fa.fa_fwd_cache(x, None, None, None, None, None, None)
    with pytest.raises(TypeError, match="k_out"):
        fa.fa_cache_read(None, None, None, None, None)
    with pytest.raises(ValueError, match=r"\[B, H, N, D\]"):
        fa.rope(x[0], None, pos, axes)
    with pytest.raises(ValueError, match="CUDA"):
        fa.KVCache8.empty(2, 2, 32, 32, device="cpu")
    with pytest.raises(TypeError, match="e4m3"):
        fa.KVCache8(x, x, x, x)
