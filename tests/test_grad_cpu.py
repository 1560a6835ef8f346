"""Refusals of the norm with rotary positions and of the gradients without a GPU, all
of them before any CUDA call, and the index arithmetic of the attention's gradient."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import unet_fa_fwd_gb300 as fa
from unet_fa_fwd_gb300 import _build
from unet_fa_fwd_gb300.binding import FaMask, FaNorm, FaRopeAxes, FaTensor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "unet_fa_fwd_gb300", "csrc")
FAR = [i << 44 for i in range(1, 20)]  # addresses of buffers that do not meet


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


# ---- fa_norm_rope, fa_norm_rope_bwd ----

def _norm(lib, back, axes=((16, 56, 56), 10000.0, 1.0), pos=FAR[0], pos_b=0, wq=FAR[10], wk=FAR[11], w_dtype=2,
          eps=1e-6, no_norm=False, no_k=False, Hq=4, Hk=2, B=2, N=10, D=128, dtype=0, pairing=0, dwq=FAR[12],
          dwk=FAR[13], ws=FAR[14], ws_bytes=1 << 30, **t):
    """t: q, k, qo, ko (results), dq, dk (gradients of the outputs) as (pointer, strides)."""
    dims, theta, scale = axes
    a = FaRopeAxes(count=len(dims))
    a.dims[:len(dims)], a.theta[:len(dims)], a.scale[:len(dims)] = dims, (theta,) * len(dims), (scale,) * len(dims)
    heads = dict(q=Hq, qo=Hq, dq=Hq, k=Hk, ko=Hk, dk=Hk)
    at = {}
    for i, (name, H) in enumerate(heads.items()):
        base = (FAR[1 + i], H * N * D, N * D, D)
        v = t.get(name, base)
        at[name] = None if v is None or (no_k and "k" in name) else ctypes.byref(FaTensor(*v))
    norm = None if no_norm else ctypes.byref(FaNorm(wq, None if no_k else wk, w_dtype, eps))
    if back:
        return lib.fa_norm_rope_bwd(ctypes.byref(a), norm, pos, pos_b, at["dq"], at["q"], at["qo"], Hq, at["dk"],
                                    at["k"], at["ko"], Hk, dwq, None if no_k else dwk, B, N, D, dtype, pairing, ws,
                                    ws_bytes, None)
    return lib.fa_norm_rope(ctypes.byref(a), norm, pos, pos_b, at["q"], at["qo"], Hq, at["k"], at["ko"], Hk, B, N, D,
                            dtype, pairing, None)


S = (4 * 10 * 128, 10 * 128, 128)      # contiguous strides of q
PACKED = (10 * 8 * 128, 128, 8 * 128)  # a token-major buffer of 8 heads


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(no_norm=True), 1), (dict(pos=None), 1), (dict(q=None), 1), (dict(q=(None, *S)), 1), (dict(qo=None), 1),
    (dict(k=None), 1), (dict(ko=None), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(Hq=0), 1), (dict(Hk=0), 1),
    (dict(D=48), 2), (dict(dtype=3), 2), (dict(pairing=2), 1), (dict(w_dtype=1), 2), (dict(w_dtype=3), 2),
    (dict(eps=-1e-6), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(axes=((16, 56), 1e4, 1.0)), 1), (dict(axes=((15, 57, 56), 1e4, 1.0)), 1),
    (dict(axes=((16, 56, 56), -1.0, 1.0)), 1), (dict(axes=((16, 56, 56), 1e4, math.nan)), 1),
    (dict(pos=FAR[0] + 2), 1), (dict(pos_b=-1), 1),
    (dict(wq=FAR[10] + 2), 1),                              # half an fp32 weight
    (dict(q=(FAR[1] + 1, *S)), 1), (dict(q=(FAR[1], -S[0], S[1], S[2])), 1), (dict(q=(FAR[1], 1 << 61, 1, 1)), 1),
    (dict(qo=(FAR[2], S[0], 0, S[2])), 1), (dict(qo=(FAR[2], S[0], S[1], 64)), 1),  # written twice
    (dict(qo=(FAR[1] + 256, *S)), 1),                       # one row behind its input
    (dict(ko=(FAR[2], *S)), 1),                             # two results in one place
    (dict(qo=(FAR[0] - 64, *S)), 1),                        # positions inside the result
    (dict(qo=(FAR[10] - 64, *S)), 1), (dict(ko=(FAR[10] - 64, *S)), 1),  # weights inside a result
])
def test_norm_rope_refusals(lib, back, kw, code):
    assert _norm(lib, back, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dq=None), 1), (dict(dk=None), 1), (dict(dq=(FAR[3] + 1, *S)), 1), (dict(dq=(FAR[2] + 256, *S)), 1),
    (dict(dwq=None), 1), (dict(dwk=None), 1), (dict(wq=None), 1), (dict(dwq=FAR[12] + 2), 1),
    (dict(dwk=FAR[12] + 256), 1),                           # the weights' gradients meet
    (dict(ws=None), 1), (dict(ws=FAR[14] + 8), 1), (dict(ws_bytes=1024), 1),
    (dict(ws=FAR[12] - 4096), 1), (dict(ws=FAR[1]), 1), (dict(ws=FAR[2]), 1), (dict(ws=FAR[3]), 1),
    (dict(dwq=FAR[1]), 1), (dict(dwq=FAR[2]), 1), (dict(dwq=FAR[10]), 1), (dict(dwq=FAR[0]), 1),
    (dict(no_k=True, dwk=FAR[13], wk=None, wq=FAR[10], Hq=0), 1),
])
def test_norm_rope_bwd_refusals(lib, kw, code):
    assert _norm(lib, True, **kw) == code


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw", [
    {}, dict(no_k=True), dict(qo=(FAR[1], *S)), dict(q=(FAR[1], *PACKED), k=(FAR[1] + 4 * 256, *PACKED)),
    dict(q=(FAR[1], 0, 0, 0)), dict(q=(FAR[1] + 2, *S)), dict(w_dtype=0), dict(wq=FAR[10] + 2, w_dtype=0),
    dict(wq=None, wk=None, dwq=None, dwk=None, ws=None, ws_bytes=0), dict(dtype=2, pairing=1), dict(eps=0.0),
])
def test_norm_rope_accepts(lib, back, kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _norm(lib, back, **kw) == 3   # the first CUDA call


def test_norm_rope_workspace(lib):
    assert fa.norm_rope_workspace_bytes(128) == 1024 * 2 * 128 * 4
    assert fa.norm_rope_workspace_bytes(48) == 0


def test_norm_rope_python_refusals():
    q = torch.zeros(1, 2, 3, 64)
    pos = torch.zeros(3, 3, dtype=torch.int32)
    axes = fa.RopeAxes((16, 24, 24))
    with pytest.raises(ValueError, match="CUDA"):
        fa.norm_rope(q, None, pos, axes)
    with pytest.raises(ValueError, match="CUDA"):
        fa.norm_rope_bwd(q, None, q, None, pos, axes)
    with pytest.raises(TypeError, match="q_out"):
        fa.fa_norm_rope(q, None, pos, axes, None, None, None, None)
    with pytest.raises(TypeError, match="dq"):
        fa.fa_norm_rope_bwd(q, None, q, None, pos, axes, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="together"):
        fa.fa_norm_rope(q, None, pos, axes, None, None, q, q)
    with pytest.raises(ValueError, match="B, H, N, D"):
        fa.norm_rope(q[0], None, pos, axes)


# ---- fa_bwd ----

def test_bwd_plan_matches_enumeration(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "bwd_geom_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe), os.path.join(HERE, "bwd_geom_check.cpp")],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr


def _bwd(lib, B=2, Hq=4, Hk=2, Nq=200, Nk=300, D=128, scale=0.1, lse=FAR[8], dlse=FAR[9], mask=None, causal=0,
         ws=FAR[10], ws_bytes=None, **t):
    """t: dout, q, k, v, out, dq, dk, dv as (pointer, strides), or None."""
    side = dict(dout=(Hq, Nq), q=(Hq, Nq), k=(Hk, Nk), v=(Hk, Nk), out=(Hq, Nq), dq=(Hq, Nq), dk=(Hk, Nk), dv=(Hk, Nk))
    at = {}
    for i, (name, (H, N)) in enumerate(side.items()):
        v = t.get(name, (FAR[i], H * N * D, N * D, D))
        at[name] = None if v is None else ctypes.byref(FaTensor(*v))
    m = None if mask is None else ctypes.byref(FaMask(*mask))
    if ws_bytes is None:
        ws_bytes = 1 << 40
    return lib.fa_bwd(at["dout"], at["q"], at["k"], at["v"], at["out"], lse, dlse, m, causal, at["dq"], at["dk"],
                      at["dv"], B, Hq, Hk, Nq, Nk, D, scale, ws, ws_bytes, None)


Q = (4 * 200 * 128, 200 * 128, 128)  # contiguous strides of q, and of k
K = (2 * 300 * 128, 300 * 128, 128)
QN = 2 * 4 * 200 * 128 * 2           # bytes of q, and of k
KN = 2 * 2 * 300 * 128 * 2


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, 1) for n in ("dout", "q", "k", "v", "out", "dq", "dk", "dv")],
    *[({n: (None, *Q)}, 1) for n in ("dout", "q", "out", "dq")],
    *[({n: (FAR[12] + 8, *Q)}, 1) for n in ("dout", "q", "out", "dq")],     # rows off 16 bytes
    *[({n: (FAR[12], *K[:2], 132)}, 1) for n in ("k", "v", "dk", "dv")],
    *[({n: (FAR[12], *K[:2], 0)}, 1) for n in ("k", "v", "dk", "dv")],      # broadcast
    *[({n: (FAR[12], Q[0], 0, Q[2])}, 1) for n in ("dout", "q", "out", "dq")],
    (dict(q=(FAR[12], -Q[0], *Q[1:])), 1), (dict(k=(FAR[12], 1 << 39, *K[1:])), 1),
    (dict(dq=(FAR[12], *Q[:2], 64)), 1), (dict(dk=(FAR[12], K[0], 128 * 299, 128)), 1),   # written twice
    (dict(lse=None), 1), (dict(lse=FAR[8] + 2), 1), (dict(dlse=FAR[9] + 2), 1),
    (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hk=0), 1), (dict(Nq=0), 1), (dict(Nk=0), 1), (dict(Hq=3), 1),
    (dict(D=48), 2), (dict(D=256), 2), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(Nq=(1 << 30) + 1), 1), (dict(B=1 << 28), 1),
    (dict(mask=(7, FAR[11], 1)), 1), (dict(mask=(1, None, 1)), 1), (dict(mask=(2, FAR[11], 2)), 1),
    (dict(mask=(3, FAR[11], 0)), 1), (dict(mask=(2, FAR[11] + 2, 1)), 1), (dict(mask=(1, FAR[11] + 2, 1)), 1),
    (dict(ws=None), 1), (dict(ws=FAR[10] + 8), 1), (dict(ws_bytes=1 << 10), 1),
    *[(dict(ws=FAR[i] - 4096), 1) for i in range(10)],                       # the workspace meets a tensor
    (dict(mask=(3, FAR[10] + 64, 1)), 1),
    (dict(dq=(FAR[1], *Q)), 1), (dict(dq=(FAR[0], *Q)), 1), (dict(dk=(FAR[2], *K)), 1), (dict(dv=(FAR[6], *K)), 1),
    (dict(dq=(FAR[2] + KN - 256, *Q)), 1), (dict(dk=(FAR[5] + QN - 256, *K)), 1), (dict(dv=(FAR[8], *K)), 1),
    (dict(dk=(FAR[9] + 16, *K)), 1), (dict(dq=(FAR[11] + 16, *Q), mask=(1, FAR[11], 1)), 1),
])
def test_bwd_refusals(lib, kw, code):
    assert _bwd(lib, **kw) == code


TOKEN = (200 * 4 * 128, 128, 4 * 128)


@pytest.mark.parametrize("kw", [
    {}, dict(dlse=None), dict(causal=1), dict(Hk=4), dict(Hk=1), dict(scale=0.0), dict(mask=(0, None, 1)),
    dict(mask=(1, FAR[11], 5)), dict(mask=(2, FAR[11] + 4, 4)), dict(mask=(3, FAR[11] + 1, 1)),
    dict(q=(FAR[1], *TOKEN), dout=(FAR[0], *TOKEN), dq=(FAR[5], *TOKEN)),
    dict(k=(FAR[2], 300 * 4 * 128, 128, 512), v=(FAR[2] + 512, 300 * 4 * 128, 128, 512)),
    dict(dk=(FAR[6], 300 * 4 * 128, 128, 512), dv=(FAR[6] + 512, 300 * 4 * 128, 128, 512)),
    dict(B=1, q=(FAR[1], 3, *Q[1:])),                                         # the stride of an axis of size 1
    dict(out=(FAR[0], *Q)),                                                   # two inputs in one place
])
def test_bwd_accepts(lib, kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _bwd(lib, **kw) == 3   # the first CUDA call


def test_bwd_workspace(lib):
    rows = 2 * 4 * 256  # whole tiles of queries
    plain = 2 * rows * 4 + 2 * 192 * 3 * 128 * 128 * 4 + 256  # (the last for the key tiles of a padding mask)
    assert fa.bwd_workspace_bytes(2, 4, 2, 200, 300, 128) == plain
    for heads in (1, 4):  # a boolean mask's bits, by rows of 3 key tiles and by keys of 2 query tiles
        bits = sum(-(-2 * heads * n // 256) * 256 for n in (200 * 3 * 16, 300 * 2 * 16))
        # ... and the tiles with a kept pair: 4 bytes each, then as bits by either side
        bits += sum(-(-2 * heads * n // 256) * 256 for n in (2 * 3 * 4, 3 * 4)) + 256 - 256
        bits += -(-2 * heads * 2 * 4 // 256) * 256
        assert fa.bwd_workspace_bytes(2, 4, 2, 200, 300, 128, heads) == plain - 256 + bits
    assert fa.bwd_workspace_bytes(2, 4, 2, 200, 300, 128, 3) == 0
    assert fa.bwd_workspace_bytes(2, 4, 2, 200, 300, 128, -1) == 0
    assert fa.bwd_workspace_bytes(2, 3, 2, 200, 300, 128) == 0
    assert fa.bwd_workspace_bytes(2, 4, 2, 200, 300, 48) == 0
    assert fa.bwd_workspace_bytes(0, 4, 2, 200, 300, 128) == 0


def test_bwd_python_refusals():
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 3)
    with pytest.raises(ValueError, match="CUDA"):
        fa.bwd(q, q, q, q, q, lse)
    with pytest.raises(ValueError, match="B, H, N, D"):
        fa.bwd(q[0], q[0], q, q, q, lse)
    with pytest.raises(TypeError, match="dk"):
        fa.fa_bwd(q, q, q, q, q, lse, q, None, q, lse)
    with pytest.raises(TypeError, match="workspace"):
        fa.fa_bwd(q, q, q, q, q, lse, q, q, q, None)
