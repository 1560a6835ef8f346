"""Rotary positions, the paged e4m3 key/value cache and the attention that reads
it: argument marshalling into ``include/fa.h``, as :mod:`.binding`.

A step of a model that generates chunk by chunk (or token by token)::

    q, k = fa.rope(q, k, pos, axes)                      # strided in, [B, H, N, D] out
    fa.cache_write(cache, k, v, table, held)             # N more tokens each
    out, lse = fa.fwd_cache(q, cache, table, held + N, causal=True)

Outputs and workspaces are allocated on the stream that the call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from .binding import (FA_OK, FaCache, FaRopeAxes, FaTensor, _stream_handle, load_library,
                      status_string)

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_PAIRINGS = {"adjacent": 0, "halves": 1}
_MAX_AXES = 4
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32

# A call's host time is most of a small call's, so the common case (tensors on the current device,
# its current stream) takes no context manager and reads the stream's handle directly.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


@contextlib.contextmanager
def _scope(device, stream):
    """The device current, and the stream too, so that what a call allocates belongs to that stream."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            with torch.cuda.stream(stream):
                yield


def _run(t: torch.Tensor, stream, call, *args):
    """call(*args, device index, stream handle) where a call on ``t`` and ``stream`` runs."""
    device = t.get_device()
    if device < 0:
        raise ValueError("tensors must be on a CUDA device")
    if stream is None and device == torch.cuda.current_device():
        return call(*args, device, _raw_stream(device))
    with _scope(t.device, stream):
        return call(*args, device, _raw_stream(device) if stream is None else _stream_handle(stream))


def _raise(name: str, rc: int) -> None:
    raise RuntimeError(f"{name} failed: {status_string(rc)}")


def _refuse(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _exact(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> int:
    """A contiguous tensor's pointer, checked."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        _refuse(t, name, dtype, shape, device)
    return t.data_ptr()


def _given(out: torch.Tensor | None, name: str) -> None:
    if out is None:
        raise TypeError(f"{name} must be a tensor")


# Four fa_tensor structs side by side (pointer and three strides each).
_Tensors = ctypes.c_longlong * 16
_SIZE = ctypes.sizeof(FaTensor)


def _strided(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> tuple:
    """A [B, H, N, D] tensor of any strides, the last axis contiguous: the fields of its fa_tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _refuse(t, name, dtype, shape, device)
    b, h, n, d = t.stride()
    if d != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return t.data_ptr(), b, h, n


class RopeAxes:
    """The axes of rotary positions: ``dims[a]`` (even) of the head dimension belong to axis a, in
    order, and sum to it.  ``theta`` and ``scale`` (which multiplies the positions) are one number
    for all axes, or one for each."""

    def __init__(self, dims, theta=10000.0, scale=1.0):
        self.dims = tuple(int(d) for d in dims)
        n = len(self.dims)
        if not 1 <= n <= _MAX_AXES:
            raise ValueError(f"1 to {_MAX_AXES} axes are supported, got {n}")
        self.theta = self._each(theta, n, "theta")
        self.scale = self._each(scale, n, "scale")
        vals = self.struct = FaRopeAxes(count=n)
        vals.dims[:n], vals.theta[:n], vals.scale[:n] = self.dims, self.theta, self.scale
        self.ref = ctypes.byref(vals)

    @staticmethod
    def _each(x, n, name):
        x = tuple(float(v) for v in x) if isinstance(x, (tuple, list)) else (float(x),) * n
        if len(x) != n:
            raise ValueError(f"{name} must be one number or one for each of the {n} axes")
        return x

    def __repr__(self):
        return f"RopeAxes(dims={self.dims}, theta={self.theta}, scale={self.scale})"


def _bhnd(t: torch.Tensor, name: str) -> tuple:
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, N, D]")
    return t.shape


def _rope_new(shape, dtype, device, token_major) -> torch.Tensor:
    B, H, N, D = shape
    if token_major:
        return torch.empty((B, N, H, D), dtype=dtype, device=device).transpose(1, 2)
    return torch.empty(shape, dtype=dtype, device=device)


def _rope(q, k, pos, axes, q_out, k_out, new, token_major, pairing, inverse, device, handle):
    B, Hq, N, D = shape = _bhnd(q, "q")
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"q must be bf16, fp16 or fp32, got {dtype}")
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {tuple(_PAIRINGS)}, got {pairing!r}")
    A = len(axes.dims)
    if pos.dtype is not _I32:
        raise TypeError(f"pos must be torch.int32, got {pos.dtype}")
    if pos.shape != (B, N, A) and pos.shape != (N, A):
        raise ValueError(f"pos must have shape {(B, N, A)} or {(N, A)}, got {tuple(pos.shape)}")
    ps = pos.stride()
    if (A > 1 and ps[-1] != 1) or (N > 1 and ps[-2] != A):
        raise ValueError("pos must be contiguous along its tokens and axes")
    if pos.get_device() != device:
        raise ValueError(f"pos must be on cuda:{device}, got {pos.device}")
    fields = _strided(q, "q", dtype, shape, device)
    if k is not None:
        Hk = _bhnd(k, "k")[1]
        k_shape = (B, Hk, N, D)
        kf = _strided(k, "k", dtype, k_shape, device)
    if new:
        q_out = _rope_new(shape, dtype, q.device, token_major)
        fields += (q_out.data_ptr(), *q_out.stride()[:3])
    else:
        fields += _strided(q_out, "q_out", dtype, shape, device)
    if k is None:
        Hk = 0
        ts = _Tensors(*fields)
        at = ctypes.addressof(ts)
        kt = ko = None
    else:
        fields += kf
        if new:
            k_out = _rope_new(k_shape, dtype, q.device, token_major)
            fields += (k_out.data_ptr(), *k_out.stride()[:3])
        else:
            fields += _strided(k_out, "k_out", dtype, k_shape, device)
        ts = _Tensors(*fields)
        at = ctypes.addressof(ts)
        kt, ko = at + 2 * _SIZE, at + 3 * _SIZE
    rc = load_library().fa_rope(axes.ref, pos.data_ptr(), ps[0] if len(ps) == 3 else 0, at, at + _SIZE, Hq, kt, ko, Hk,
                                B, N, D, _DTYPES[dtype], _PAIRINGS[pairing], inverse, handle)
    if rc != FA_OK:
        _raise("fa_rope", rc)
    return q_out, k_out


def fa_rope(q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor, axes: RopeAxes, q_out: torch.Tensor,
            k_out: torch.Tensor | None, pairing: str = "adjacent", inverse: bool = False, stream=None) -> None:
    """Enqueue the rotation into caller-provided outputs (any strides; the inputs themselves for in
    place).  q [B, Hq, N, D] and k [B, Hk, N, D] (or None) of one dtype, bf16, fp16 or fp32; pos int32
    [B, N, A] or [N, A]."""
    _given(q_out, "q_out")
    if (k is None) != (k_out is None):
        raise ValueError("pass k and k_out together, or neither")
    _run(q, stream, _rope, q, k, pos, axes, q_out, k_out, False, False, pairing, bool(inverse))


def rope(q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor, axes: RopeAxes, pairing: str = "adjacent",
         inverse: bool = False, token_major: bool = False, stream=None):
    """Allocate outputs and turn q and k (k may be None) by their positions; returns (q, k),
    contiguous [B, H, N, D] as the attention takes them, or with ``token_major`` views of contiguous
    [B, N, H, D] tensors.  Inputs may have any strides (slices of a projection).  Autograd does not
    record the call: the gradients are :func:`rope_bwd`'s."""
    _bhnd(q, "q")
    return _run(q, stream, _rope, q, k, pos, axes, None, None, True, token_major, pairing, bool(inverse))


def rope_bwd(dq: torch.Tensor, dk: torch.Tensor | None, pos: torch.Tensor, axes: RopeAxes,
             pairing: str = "adjacent", token_major: bool = False, stream=None):
    """Gradients of :func:`rope` with respect to q and k, from those of its outputs (the inverse
    rotation); ``token_major`` as there."""
    return rope(dq, dk, pos, axes, pairing=pairing, inverse=True, token_major=token_major, stream=stream)


class KVCache8:
    """A paged key/value cache in e4m3: codes ``k``, ``v`` [pages, H, page_tokens, D]
    (torch.float8_e4m3fn or uint8) and their scales ``k_scale``, ``v_scale`` fp32 [pages, H], one for
    each page and head, powers of two.  Nothing needs clearing; which pages a sequence owns is the
    caller's table."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if k.dim() != 4:
            raise ValueError("k must be [pages, H, page_tokens, D]")
        pages, H, page, D = k.shape
        dtype, device = k.dtype, k.get_device()
        if dtype is not torch.float8_e4m3fn and dtype is not torch.uint8:
            raise TypeError(f"k must be torch.float8_e4m3fn or torch.uint8, got {dtype}")
        if device < 0:
            raise ValueError("k must be a CUDA tensor")
        self.struct = FaCache(_exact(k, "k", dtype, k.shape, device), _exact(v, "v", dtype, k.shape, device),
                              _exact(k_scale, "k_scale", _F32, (pages, H), device),
                              _exact(v_scale, "v_scale", _F32, (pages, H), device), pages, H, page, D)
        self.ref = ctypes.byref(self.struct)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.heads, self.page_tokens, self.head_dim = H, page, D

    @classmethod
    def empty(cls, num_pages: int, heads: int, page_tokens: int, head_dim: int, device="cuda") -> "KVCache8":
        codes = [torch.empty((num_pages, heads, page_tokens, head_dim), dtype=torch.uint8, device=device)
                 .view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.empty((num_pages, heads), dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales)


def _table(table: torch.Tensor, B: int, device: int) -> int:
    if table.dim() != 2:
        raise ValueError("table must be [B, pages of a sequence]")
    return _exact(table, "table", _I32, (B, table.shape[1]), device)


def _ints(t: torch.Tensor | None, name: str, B: int, device: int) -> int | None:
    return None if t is None else _exact(t, name, _I32, (B,), device)


def _same_heads(cache: KVCache8, name: str, H: int, D: int) -> None:
    if H != cache.heads or D != cache.head_dim:
        raise ValueError(f"{name} must have {cache.heads} heads of {cache.head_dim}, got {H} of {D}")


def _write(cache, k, v, table, start, count, device, handle):
    B, H, N, D = shape = _bhnd(k, "k")
    _same_heads(cache, "k", H, D)
    ts = _Tensors(*_strided(k, "k", _BF16, shape, device), *_strided(v, "v", _BF16, shape, device))
    at = ctypes.addressof(ts)
    rc = load_library().fa_cache_write(cache.ref, at, at + _SIZE, _table(table, B, device), table.shape[1],
                                       _ints(start, "start", B, device), _ints(count, "count", B, device), B, N,
                                       handle)
    if rc != FA_OK:
        _raise("fa_cache_write", rc)


def cache_write(cache: KVCache8, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, start: torch.Tensor,
                count: torch.Tensor | None = None, stream=None) -> None:
    """Quantise tokens and append them: token i < count[b] (N if None) of k, v (bf16 [B, H, N, D], any
    strides) goes to position start[b] + i of sequence b, page table[b, position // page_tokens].
    start int32 [B] is what each sequence holds already.  The pages written must be distinct."""
    _run(cache.k, stream, _write, cache, k, v, table, start, count)


def _read(cache, table, lens, k_out, v_out, n, start, device, handle):
    if k_out is None:
        B, N = table.shape[0], n
        shape = (B, cache.heads, N, cache.head_dim)
        k_out = torch.empty(shape, dtype=_BF16, device=cache.k.device)
        v_out = torch.empty(shape, dtype=_BF16, device=cache.k.device)
        kp, vp = k_out.data_ptr(), v_out.data_ptr()
    else:
        B, H, N, D = shape = _bhnd(k_out, "k_out")
        _same_heads(cache, "k_out", H, D)
        kp = _exact(k_out, "k_out", _BF16, shape, device)
        vp = _exact(v_out, "v_out", _BF16, shape, device)
    rc = load_library().fa_cache_read(cache.ref, _table(table, B, device), table.shape[1],
                                      _ints(lens, "lens", B, device), _ints(start, "start", B, device), kp, vp, B, N,
                                      handle)
    if rc != FA_OK:
        _raise("fa_cache_read", rc)
    return k_out, v_out


def fa_cache_read(cache: KVCache8, table: torch.Tensor, lens: torch.Tensor, k_out: torch.Tensor,
                  v_out: torch.Tensor, start: torch.Tensor | None = None, stream=None) -> None:
    """Read tokens start[b] (0 if None) .. start[b] + N - 1 of each sequence into caller-provided bf16
    [B, H, N, D]; positions from lens[b] on give zeros."""
    _given(k_out, "k_out")
    _run(cache.k, stream, _read, cache, table, lens, k_out, v_out, None, start)


def cache_read(cache: KVCache8, table: torch.Tensor, lens: torch.Tensor, n: int,
               start: torch.Tensor | None = None, stream=None):
    """Allocate outputs and read ``n`` tokens of each sequence back; returns (k, v) bf16 [B, H, n, D]."""
    return _run(cache.k, stream, _read, cache, table, lens, None, None, n, start)


def cache_workspace_bytes(B: int, Hq: int, Hk: int, Nq: int, D: int, table_width: int, page_tokens: int) -> int:
    return int(load_library().fa_cache_workspace_bytes(B, Hq, Hk, Nq, D, table_width, page_tokens))


def _attend(q, cache, table, lens, out, lse, workspace, causal, q_start, scale, device, handle):
    B, Hq, Nq, D = shape = _bhnd(q, "q")
    if D != cache.head_dim:
        raise ValueError(f"q must have heads of {cache.head_dim}, got {D}")
    qp, tab = _exact(q, "q", _BF16, shape, device), _table(table, B, device)
    lib = load_library()
    if out is None:
        need = lib.fa_cache_workspace_bytes(B, Hq, cache.heads, Nq, D, table.shape[1], cache.page_tokens)
        out = torch.empty_like(q)
        lse = torch.empty((B, Hq, Nq), dtype=_F32, device=q.device)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        op, lp = out.data_ptr(), lse.data_ptr()
    else:
        op = _exact(out, "out", _BF16, shape, device)
        lp = _exact(lse, "lse", _F32, (B, Hq, Nq), device)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.get_device() != device:
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    rc = lib.fa_fwd_cache(qp, cache.ref, tab, table.shape[1], _ints(lens, "lens", B, device),
                          _ints(q_start, "q_start", B, device), causal, op, lp, B, Hq, Nq, scale, ws_ptr, ws_bytes,
                          handle)
    if rc != FA_OK:
        _raise("fa_fwd_cache", rc)
    return out, lse


def fa_fwd_cache(q: torch.Tensor, cache: KVCache8, table: torch.Tensor, lens: torch.Tensor, out: torch.Tensor,
                 lse: torch.Tensor, workspace: torch.Tensor | None, causal: bool = False,
                 q_start: torch.Tensor | None = None, scale: float | None = None, stream=None) -> None:
    """Enqueue the attention to the cache into caller-provided ``out`` and ``lse``; ``workspace`` holds
    at least cache_workspace_bytes(...) bytes (None when that is 0)."""
    _given(out, "out")
    _run(cache.k, stream, _attend, q, cache, table, lens, out, lse, workspace, bool(causal), q_start, scale)


def fwd_cache(q: torch.Tensor, cache: KVCache8, table: torch.Tensor, lens: torch.Tensor, causal: bool = False,
              q_start: torch.Tensor | None = None, scale: float | None = None, stream=None):
    """Allocate outputs and workspace and attend to the cache: q bf16 [B, Hq, Nq, D] against the keys
    0 .. lens[b] - 1 of each sequence (int32 [B]); with ``causal`` row i sees the keys up to
    q_start[b] + i (lens[b] - Nq + i if None).  Returns (O bf16 [B, Hq, Nq, D], LSE fp32 [B, Hq, Nq])."""
    return _run(cache.k, stream, _attend, q, cache, table, lens, None, None, None, bool(causal), q_start, scale)
