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


@contextlib.contextmanager
def _scope(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            with torch.cuda.stream(stream):
                yield


def _on(t: torch.Tensor, stream):
    """Where a call on ``t`` runs: its device current, and ``stream`` (the device's current
    stream if None) current, so that what the call allocates belongs to that stream."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if stream is None and t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return _scope(t.device, stream)


def _raise(name: str, rc: int) -> None:
    if rc != FA_OK:
        raise RuntimeError(f"{name} failed: {status_string(rc)}")


def _same_device(t: torch.Tensor, name: str, other: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != other.device:
        raise ValueError(f"{name} must be on {other.device}, got {t.device}")


def _exact(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, like: torch.Tensor) -> int:
    """A contiguous tensor's pointer, checked."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _same_device(t, name, like)
    return t.data_ptr()


def _strided(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, like: torch.Tensor) -> FaTensor:
    """A [B, H, N, D] tensor of any strides, the last axis contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    b, h, n, d = t.stride()
    if d != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    _same_device(t, name, like)
    return FaTensor(t.data_ptr(), b, h, n)


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
    return tuple(t.shape)


def fa_rope(q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor, axes: RopeAxes, q_out: torch.Tensor,
            k_out: torch.Tensor | None, pairing: str = "adjacent", inverse: bool = False, stream=None) -> None:
    """Enqueue the rotation into caller-provided outputs (any strides; the inputs themselves for in
    place).  q [B, Hq, N, D] and k [B, Hk, N, D] (or None) of one dtype, bf16, fp16 or fp32; pos int32
    [B, N, A] or [N, A]."""
    B, Hq, N, D = _bhnd(q, "q")
    if q.dtype not in _DTYPES:
        raise TypeError(f"q must be bf16, fp16 or fp32, got {q.dtype}")
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {tuple(_PAIRINGS)}, got {pairing!r}")
    if (k is None) != (k_out is None):
        raise ValueError("pass k and k_out together, or neither")
    A = len(axes.dims)
    if pos.dtype != torch.int32:
        raise TypeError(f"pos must be torch.int32, got {pos.dtype}")
    if pos.shape != (B, N, A) and pos.shape != (N, A):
        raise ValueError(f"pos must have shape {(B, N, A)} or {(N, A)}, got {tuple(pos.shape)}")
    if (A > 1 and pos.stride(-1) != 1) or (N > 1 and pos.stride(-2) != A):
        raise ValueError("pos must be contiguous along its tokens and axes")
    _same_device(pos, "pos", q)
    ts = [_strided(q, "q", q.dtype, (B, Hq, N, D), q), _strided(q_out, "q_out", q.dtype, (B, Hq, N, D), q)]
    Hk = 0
    if k is not None:
        Hk = _bhnd(k, "k")[1]
        ts += [_strided(k, "k", q.dtype, (B, Hk, N, D), q), _strided(k_out, "k_out", q.dtype, (B, Hk, N, D), q)]
    refs = [ctypes.byref(t) for t in ts] + [None] * (4 - len(ts))
    with _on(q, stream):
        rc = load_library().fa_rope(ctypes.byref(axes.struct), pos.data_ptr(), pos.stride(0) if pos.dim() == 3 else 0,
                                    refs[0], refs[1], Hq, refs[2], refs[3], Hk, B, N, D, _DTYPES[q.dtype],
                                    _PAIRINGS[pairing], int(bool(inverse)), _stream_handle(stream))
    _raise("fa_rope", rc)


def _rope_new(t: torch.Tensor, token_major: bool) -> torch.Tensor:
    B, H, N, D = t.shape
    if token_major:
        return torch.empty((B, N, H, D), dtype=t.dtype, device=t.device).transpose(1, 2)
    return torch.empty((B, H, N, D), dtype=t.dtype, device=t.device)


def rope(q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor, axes: RopeAxes, pairing: str = "adjacent",
         inverse: bool = False, token_major: bool = False, stream=None):
    """Allocate outputs and turn q and k (k may be None) by their positions; returns (q, k),
    contiguous [B, H, N, D] as the attention takes them, or with ``token_major`` views of contiguous
    [B, N, H, D] tensors.  Inputs may have any strides (slices of a projection)."""
    _bhnd(q, "q")
    if k is not None:
        _bhnd(k, "k")
    with _on(q, stream):
        q_out = _rope_new(q, token_major)
        k_out = None if k is None else _rope_new(k, token_major)
    fa_rope(q, k, pos, axes, q_out, k_out, pairing=pairing, inverse=inverse, stream=stream)
    return q_out, k_out


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
        if k.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError(f"k must be torch.float8_e4m3fn or torch.uint8, got {k.dtype}")
        self.struct = FaCache(_exact(k, "k", k.dtype, k.shape, k), _exact(v, "v", k.dtype, k.shape, k),
                              _exact(k_scale, "k_scale", torch.float32, (pages, H), k),
                              _exact(v_scale, "v_scale", torch.float32, (pages, H), k), pages, H, page, D)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale

    @classmethod
    def empty(cls, num_pages: int, heads: int, page_tokens: int, head_dim: int, device="cuda") -> "KVCache8":
        codes = [torch.empty((num_pages, heads, page_tokens, head_dim), dtype=torch.uint8, device=device)
                 .view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.empty((num_pages, heads), dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales)


def _table(table: torch.Tensor, B: int, cache: KVCache8) -> int:
    if table.dim() != 2:
        raise ValueError("table must be [B, pages of a sequence]")
    return _exact(table, "table", torch.int32, (B, table.shape[1]), cache.k)


def _ints(t: torch.Tensor | None, name: str, B: int, cache: KVCache8) -> int | None:
    return None if t is None else _exact(t, name, torch.int32, (B,), cache.k)


def cache_write(cache: KVCache8, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, start: torch.Tensor,
                count: torch.Tensor | None = None, stream=None) -> None:
    """Quantise tokens and append them: token i < count[b] (N if None) of k, v (bf16 [B, H, N, D], any
    strides) goes to position start[b] + i of sequence b, page table[b, position // page_tokens].
    start int32 [B] is what each sequence holds already.  The pages written must be distinct."""
    B, H, N, D = _bhnd(k, "k")
    c = cache.struct
    if (H, D) != (c.H, c.D):
        raise ValueError(f"k must have {c.H} heads of {c.D}, got {H} of {D}")
    kt = _strided(k, "k", torch.bfloat16, (B, H, N, D), cache.k)
    vt = _strided(v, "v", torch.bfloat16, (B, H, N, D), cache.k)
    tab, at, n = _table(table, B, cache), _ints(start, "start", B, cache), _ints(count, "count", B, cache)
    with _on(cache.k, stream):
        rc = load_library().fa_cache_write(ctypes.byref(c), ctypes.byref(kt), ctypes.byref(vt), tab, table.shape[1],
                                           at, n, B, N, _stream_handle(stream))
    _raise("fa_cache_write", rc)


def fa_cache_read(cache: KVCache8, table: torch.Tensor, lens: torch.Tensor, k_out: torch.Tensor,
                  v_out: torch.Tensor, start: torch.Tensor | None = None, stream=None) -> None:
    """Read tokens start[b] (0 if None) .. start[b] + N - 1 of each sequence into caller-provided bf16
    [B, H, N, D]; positions from lens[b] on give zeros."""
    B, H, N, D = _bhnd(k_out, "k_out")
    c = cache.struct
    if (H, D) != (c.H, c.D):
        raise ValueError(f"k_out must have {c.H} heads of {c.D}, got {H} of {D}")
    ko = _exact(k_out, "k_out", torch.bfloat16, (B, H, N, D), cache.k)
    vo = _exact(v_out, "v_out", torch.bfloat16, (B, H, N, D), cache.k)
    tab, n, at = _table(table, B, cache), _ints(lens, "lens", B, cache), _ints(start, "start", B, cache)
    with _on(cache.k, stream):
        rc = load_library().fa_cache_read(ctypes.byref(c), tab, table.shape[1], n, at, ko, vo, B, N,
                                          _stream_handle(stream))
    _raise("fa_cache_read", rc)


def cache_read(cache: KVCache8, table: torch.Tensor, lens: torch.Tensor, n: int,
               start: torch.Tensor | None = None, stream=None):
    """Allocate outputs and read ``n`` tokens of each sequence back; returns (k, v) bf16 [B, H, n, D]."""
    c = cache.struct
    with _on(cache.k, stream):
        k, v = (torch.empty((table.shape[0], c.H, n, c.D), dtype=torch.bfloat16, device=cache.k.device)
                for _ in range(2))
    fa_cache_read(cache, table, lens, k, v, start=start, stream=stream)
    return k, v


def cache_workspace_bytes(B: int, Hq: int, Hk: int, Nq: int, D: int, table_width: int, page_tokens: int) -> int:
    return int(load_library().fa_cache_workspace_bytes(B, Hq, Hk, Nq, D, table_width, page_tokens))


def fa_fwd_cache(q: torch.Tensor, cache: KVCache8, table: torch.Tensor, lens: torch.Tensor, out: torch.Tensor,
                 lse: torch.Tensor, workspace: torch.Tensor | None, causal: bool = False,
                 q_start: torch.Tensor | None = None, scale: float | None = None, stream=None) -> None:
    """Enqueue the attention to the cache into caller-provided ``out`` and ``lse``; ``workspace`` holds
    at least cache_workspace_bytes(...) bytes (None when that is 0)."""
    B, Hq, Nq, D = _bhnd(q, "q")
    c = cache.struct
    if D != c.D:
        raise ValueError(f"q must have heads of {c.D}, got {D}")
    qp = _exact(q, "q", torch.bfloat16, (B, Hq, Nq, D), cache.k)
    op = _exact(out, "out", torch.bfloat16, (B, Hq, Nq, D), cache.k)
    lp = _exact(lse, "lse", torch.float32, (B, Hq, Nq), cache.k)
    tab, n, at = _table(table, B, cache), _ints(lens, "lens", B, cache), _ints(q_start, "q_start", B, cache)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        _same_device(workspace, "workspace", q)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on(q, stream):
        rc = load_library().fa_fwd_cache(qp, ctypes.byref(c), tab, table.shape[1], n, at, int(bool(causal)), op, lp,
                                         B, Hq, Nq, ctypes.c_float(scale), ws_ptr, ws_bytes, _stream_handle(stream))
    _raise("fa_fwd_cache", rc)


def fwd_cache(q: torch.Tensor, cache: KVCache8, table: torch.Tensor, lens: torch.Tensor, causal: bool = False,
              q_start: torch.Tensor | None = None, scale: float | None = None, stream=None):
    """Allocate outputs and workspace and attend to the cache: q bf16 [B, Hq, Nq, D] against the keys
    0 .. lens[b] - 1 of each sequence (int32 [B]); with ``causal`` row i sees the keys up to
    q_start[b] + i (lens[b] - Nq + i if None).  Returns (O bf16 [B, Hq, Nq, D], LSE fp32 [B, Hq, Nq])."""
    B, Hq, Nq, D = _bhnd(q, "q")
    c = cache.struct
    need = cache_workspace_bytes(B, Hq, c.H, Nq, D, table.shape[-1], c.page_tokens)
    with _on(q, stream):
        out = torch.empty((B, Hq, Nq, D), dtype=torch.bfloat16, device=q.device)
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    fa_fwd_cache(q, cache, table, lens, out, lse, ws, causal=causal, q_start=q_start, scale=scale, stream=stream)
    return out, lse
