"""What training an attention layer needs around the forward: the attention's
gradient, and the norm of queries and keys for each head with the rotary positions
in the same pass, with its gradient: argument marshalling into ``include/fa.h``, as :mod:`.binding` and :mod:`.cache`.

Autograd records none of these calls; the gradients are calls of their own::

    q, k = fa.norm_rope(q0, k0, pos, axes, wq, wk)
    out, lse = fa.fwd(q, k, v)
    dq, dk, dv = fa.bwd(dout, q, k, v, out, lse)
    dq0, dk0, dwq, dwk = fa.norm_rope_bwd(dq, dk, q0, k0, pos, axes, wq, wk)

Outputs and workspaces are allocated on the stream that the call runs on.
"""
from __future__ import annotations

import array
import ctypes
import functools
import math

import torch

from .binding import (FA_MASK_ADDITIVE, FA_MASK_BOOL, FA_MASK_KEY_PADDING, FA_OK, FaMask, FaNorm,
                      load_library)
from .cache import (_BF16, _DTYPES, _F32, _PAIRINGS, _SIZE, RopeAxes, _bhnd, _exact, _given, _positions, _raise, _rope_new,
                    _run, _strided)


def _tensors(fields) -> tuple:
    """fa_tensor structs side by side (pointer and three strides each), which live as long as the first result, and
    their address."""
    ts = array.array("q", fields)
    return ts, ts.buffer_info()[0]


def _rope_strides(shape, token_major) -> tuple:
    """The strides of a tensor that _rope_new allocates, but for the last."""
    B, H, N, D = shape
    return (N * H * D, D, H * D) if token_major else (H * N * D, N * D, D)


def _norm(q, k, q_weight, k_weight, eps, device) -> FaNorm:
    D = q.shape[3]
    if k is None and k_weight is not None:
        raise ValueError("k_weight without k")
    given = [(w, name) for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")) if w is not None]
    dtype = given[0][0].dtype if given else _F32
    if dtype is not _F32 and dtype is not q.dtype:
        raise TypeError(f"weights must be torch.float32 or {q.dtype}, got {dtype}")
    ptr = {name: _exact(w, name, dtype, (D,), device) for w, name in given}
    return FaNorm(ptr.get("q_weight"), ptr.get("k_weight"), _DTYPES[dtype], float(eps))


def _check(q, pairing):
    shape, dtype = _bhnd(q, "q"), q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"q must be bf16, fp16 or fp32, got {dtype}")
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {tuple(_PAIRINGS)}, got {pairing!r}")
    return shape, dtype


def _side(tensors, names, shape, dtype, device, new, token_major):
    """The fa_tensor fields of inputs and an output (the last of ``tensors``; allocated if ``new``), and the
    output."""
    fields = ()
    for t, name in zip(tensors[:-1], names):
        fields += _strided(t, name, dtype, shape, device)
    out = tensors[-1]
    if new:
        out = _rope_new(shape, dtype, tensors[0].device, token_major)
        return fields + (out.data_ptr(), *_rope_strides(shape, token_major)), out
    return fields + _strided(out, names[-1], dtype, shape, device), out


def _norm_rope(q, k, pos, axes, q_weight, k_weight, eps, q_out, k_out, new, token_major, pairing, device, handle):
    shape, dtype = _check(q, pairing)
    B, Hq, N, D = shape
    pos_b = _positions(pos, B, N, len(axes.dims), device)
    norm = _norm(q, k, q_weight, k_weight, eps, device)
    fields, q_out = _side((q, q_out), ("q", "q_out"), shape, dtype, device, new, token_major)
    Hk = 0
    if k is not None:
        Hk = _bhnd(k, "k")[1]
        more, k_out = _side((k, k_out), ("k", "k_out"), (B, Hk, N, D), dtype, device, new, token_major)
        fields += more
    ts, at = _tensors(fields)
    rc = load_library().fa_norm_rope(axes.ref, ctypes.byref(norm), pos.data_ptr(), pos_b, at, at + _SIZE, Hq,
                                     at + 2 * _SIZE if k is not None else None,
                                     at + 3 * _SIZE if k is not None else None, Hk, B, N, D, _DTYPES[dtype],
                                     _PAIRINGS[pairing], handle)
    if rc != FA_OK:
        _raise("fa_norm_rope", rc)
    return q_out, k_out


def fa_norm_rope(q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor, axes: RopeAxes,
                 q_weight: torch.Tensor | None, k_weight: torch.Tensor | None, q_out: torch.Tensor,
                 k_out: torch.Tensor | None, eps: float = 1e-6, pairing: str = "adjacent", stream=None) -> None:
    """Enqueue the norm and rotation into caller-provided outputs (any strides; the inputs themselves for in
    place).  q [B, Hq, N, D] and k [B, Hk, N, D] (or None) of one dtype, bf16, fp16 or fp32; pos int32 [B, N, A]
    or [N, A]; weights [D] of that dtype or fp32, or None."""
    _given(q_out, "q_out")
    if (k is None) != (k_out is None):
        raise ValueError("pass k and k_out together, or neither")
    _run(q, stream, _norm_rope, q, k, pos, axes, q_weight, k_weight, eps, q_out, k_out, False, False, pairing)


def norm_rope(q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor, axes: RopeAxes,
              q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
              pairing: str = "adjacent", token_major: bool = False, stream=None):
    """Allocate outputs, normalise the rows of q and k (k may be None) by the root of their mean square, multiply
    by the weights and turn them by their positions, as :func:`~unet_fa_fwd_gb300.rope` does; returns (q, k).
    The gradients are :func:`norm_rope_bwd`'s."""
    _bhnd(q, "q")
    return _run(q, stream, _norm_rope, q, k, pos, axes, q_weight, k_weight, eps, None, None, True, token_major,
                pairing)


@functools.lru_cache(maxsize=1024)  # (a call of its own into the library otherwise)
def norm_rope_workspace_bytes(D: int) -> int:
    return int(load_library().fa_norm_rope_workspace_bytes(D))


def _norm_rope_bwd(dq_out, dk_out, q, k, pos, axes, q_weight, k_weight, eps, dq, dk, dwq, dwk, workspace, new,
                   token_major, pairing, device, handle):
    shape, dtype = _check(q, pairing)
    B, Hq, N, D = shape
    pos_b = _positions(pos, B, N, len(axes.dims), device)
    norm = _norm(q, k, q_weight, k_weight, eps, device)
    if (k is None) != (dk_out is None):
        raise ValueError("pass k and its gradient together, or neither")
    fields, dq = _side((dq_out, q, dq), ("dq_out", "q", "dq"), shape, dtype, device, new, token_major)
    Hk = 0
    if k is not None:
        Hk = _bhnd(k, "k")[1]
        more, dk = _side((dk_out, k, dk), ("dk_out", "k", "dk"), (B, Hk, N, D), dtype, device, new, token_major)
        fields += more
    lib = load_library()
    if new:
        dwq, dwk = (None if w is None else torch.empty(D, dtype=_F32, device=q.device) for w in (q_weight, k_weight))
        if dwq is not None or dwk is not None:
            workspace = torch.empty(norm_rope_workspace_bytes(D), dtype=torch.uint8, device=q.device)
    else:
        for w, dw, name in ((q_weight, dwq, "dq_weight"), (k_weight, dwk, "dk_weight")):
            if (w is None) != (dw is None):
                raise ValueError(f"pass {name} together with its weight, or neither")
    at_w = [None if dw is None else _exact(dw, name, _F32, (D,), device)
            for dw, name in ((dwq, "dq_weight"), (dwk, "dk_weight"))]
    ws_ptr, ws_bytes = _workspace(workspace, device)
    ts, at = _tensors(fields)
    kt = [at + i * _SIZE if k is not None else None for i in (3, 4, 5)]
    rc = lib.fa_norm_rope_bwd(axes.ref, ctypes.byref(norm), pos.data_ptr(), pos_b, at, at + _SIZE, at + 2 * _SIZE, Hq,
                              *kt, Hk, *at_w, B, N, D, _DTYPES[dtype], _PAIRINGS[pairing], ws_ptr, ws_bytes, handle)
    if rc != FA_OK:
        _raise("fa_norm_rope_bwd", rc)
    return dq, dk, dwq, dwk


def _workspace(workspace, device) -> tuple:
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous() or workspace.get_device() != device:
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def fa_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor | None, q: torch.Tensor, k: torch.Tensor | None,
                     pos: torch.Tensor, axes: RopeAxes, q_weight: torch.Tensor | None,
                     k_weight: torch.Tensor | None, dq: torch.Tensor, dk: torch.Tensor | None,
                     dq_weight: torch.Tensor | None, dk_weight: torch.Tensor | None,
                     workspace: torch.Tensor | None, eps: float = 1e-6, pairing: str = "adjacent",
                     stream=None) -> None:
    """Enqueue the gradients of :func:`fa_norm_rope` into caller-provided ``dq``, ``dk`` (any strides; ``dq_out``
    and ``dk_out``, or q and k, themselves for in place) and fp32 [D] ``dq_weight``, ``dk_weight`` (None where
    there is no weight); ``workspace`` holds norm_rope_workspace_bytes(D) bytes (None without weights)."""
    _given(dq, "dq")
    if (k is None) != (dk is None):
        raise ValueError("pass k and dk together, or neither")
    _run(q, stream, _norm_rope_bwd, dq_out, dk_out, q, k, pos, axes, q_weight, k_weight, eps, dq, dk, dq_weight,
         dk_weight, workspace, False, False, pairing)


def norm_rope_bwd(dq: torch.Tensor, dk: torch.Tensor | None, q: torch.Tensor, k: torch.Tensor | None,
                  pos: torch.Tensor, axes: RopeAxes, q_weight: torch.Tensor | None = None,
                  k_weight: torch.Tensor | None = None, eps: float = 1e-6, pairing: str = "adjacent",
                  token_major: bool = False, stream=None):
    """Gradients of :func:`norm_rope` from those of its outputs (``dq``, ``dk``) and its inputs; returns (gradient
    of q, of k, of q_weight, of k_weight), the last two fp32 [D] (None where there is no weight), the first two
    with ``token_major`` views of contiguous [B, N, H, D] tensors, as the projection ahead takes them."""
    _bhnd(q, "q")
    return _run(q, stream, _norm_rope_bwd, dq, dk, q, k, pos, axes, q_weight, k_weight, eps, None, None, None, None,
                None, True, token_major, pairing)


@functools.lru_cache(maxsize=1024)
def bwd_workspace_bytes(B: int, Hq: int, Hk: int, Nq: int, Nk: int, D: int, bool_mask_heads: int = 0) -> int:
    """``bool_mask_heads``: heads (1 or Hq) of a boolean mask, which is kept as bits; 0 for any other mask."""
    return int(load_library().fa_bwd_workspace_bytes(B, Hq, Hk, Nq, Nk, D, bool_mask_heads))


def _mask(key_mask, full_mask, B, Hq, Nq, Nk, device):
    if key_mask is not None and full_mask is not None:
        raise ValueError("pass key_mask or full_mask, not both")
    if key_mask is not None:
        return ctypes.byref(FaMask(FA_MASK_KEY_PADDING, _exact(key_mask, "key_mask", _F32, (B, Nk), device), 1))
    if full_mask is None:
        return None
    if full_mask.dim() != 4 or full_mask.shape[1] not in (1, Hq):
        raise ValueError("full_mask must be [B, 1|Hq, Nq, Nk]")
    if full_mask.dtype not in (_F32, torch.bool, torch.uint8):
        raise TypeError("full_mask must be float32 (additive) or bool/uint8")
    heads = full_mask.shape[1]
    at = _exact(full_mask, "full_mask", full_mask.dtype, (B, heads, Nq, Nk), device)
    return ctypes.byref(FaMask(FA_MASK_ADDITIVE if full_mask.dtype is _F32 else FA_MASK_BOOL, at, heads))


def _bwd(dout, q, k, v, out, lse, dlse, key_mask, full_mask, causal, scale, dq, dk, dv, workspace, new, token_major,
         device, handle):
    B, Hq, Nq, D = q_shape = _bhnd(q, "q")
    Hk, Nk = _bhnd(k, "k")[1:3]
    k_shape = (B, Hk, Nk, D)
    fields = ()
    for t, name, shape in ((dout, "dout", q_shape), (q, "q", q_shape), (k, "k", k_shape), (v, "v", k_shape),
                           (out, "out", q_shape)):
        fields += _strided(t, name, _BF16, shape, device)
    lib = load_library()
    if new:
        on = q.device
        dq, dk, dv = (_rope_new(q_shape, _BF16, on, token_major), _rope_new(k_shape, _BF16, on, token_major),
                      _rope_new(k_shape, _BF16, on, token_major))
        heads = 0 if full_mask is None or full_mask.dtype is _F32 or full_mask.dim() != 4 else full_mask.shape[1]
        workspace = torch.empty(bwd_workspace_bytes(B, Hq, Hk, Nq, Nk, D, heads), dtype=torch.uint8, device=on)
        q_strides, k_strides = _rope_strides(q_shape, token_major), _rope_strides(k_shape, token_major)
        fields += (dq.data_ptr(), *q_strides, dk.data_ptr(), *k_strides, dv.data_ptr(), *k_strides)
    else:
        for t, name, shape in ((dq, "dq", q_shape), (dk, "dk", k_shape), (dv, "dv", k_shape)):
            fields += _strided(t, name, _BF16, shape, device)
    lse_at = _exact(lse, "lse", _F32, (B, Hq, Nq), device)
    dlse_at = None if dlse is None else _exact(dlse, "dlse", _F32, (B, Hq, Nq), device)
    ws_ptr, ws_bytes = _workspace(workspace, device)
    ts, at = _tensors(fields)
    rc = lib.fa_bwd(at, at + _SIZE, at + 2 * _SIZE, at + 3 * _SIZE, at + 4 * _SIZE, lse_at, dlse_at,
                    _mask(key_mask, full_mask, B, Hq, Nq, Nk, device), causal, at + 5 * _SIZE, at + 6 * _SIZE,
                    at + 7 * _SIZE, B, Hq, Hk, Nq, Nk, D,
                    1.0 / math.sqrt(D) if scale is None else scale, ws_ptr, ws_bytes, handle)
    if rc != FA_OK:
        _raise("fa_bwd", rc)
    return dq, dk, dv


def fa_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
           lse: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, workspace: torch.Tensor,
           key_mask: torch.Tensor | None = None, full_mask: torch.Tensor | None = None, causal: bool = False,
           scale: float | None = None, dlse: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue the attention's gradient into caller-provided ``dq``, ``dk``, ``dv`` (any strides whose rows start
    16-byte aligned); ``workspace`` holds bwd_workspace_bytes(...) bytes."""
    for t, name in ((dq, "dq"), (dk, "dk"), (dv, "dv"), (workspace, "workspace")):
        _given(t, name)
    _run(q, stream, _bwd, dout, q, k, v, out, lse, dlse, key_mask, full_mask, bool(causal), scale, dq, dk, dv,
         workspace, False, False)


def bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
        key_mask: torch.Tensor | None = None, full_mask: torch.Tensor | None = None, causal: bool = False,
        scale: float | None = None, dlse: torch.Tensor | None = None, token_major: bool = False, stream=None):
    """Allocate outputs and workspace and compute the gradients of :func:`~unet_fa_fwd_gb300.fwd` and
    :func:`~unet_fa_fwd_gb300.fwd_ex` from what they were given and returned: ``dout`` (and ``dlse``) are the
    gradients of O (and LSE).  bf16 [B, H, N, D] tensors of any strides whose rows start 16-byte aligned; k and v
    may have fewer heads than q (shared by neighbouring query heads, whose gradients add up).  Masks as
    fwd_ex's, of any finite size; rows that see no key may hold anything.  Returns (dq, dk, dv), contiguous or
    with ``token_major`` views of contiguous [B, N, H, D] tensors.  Autograd does not record the call."""
    _bhnd(q, "q")
    return _run(q, stream, _bwd, dout, q, k, v, out, lse, dlse, key_mask, full_mask, bool(causal), scale, None, None,
                None, None, True, token_major)
