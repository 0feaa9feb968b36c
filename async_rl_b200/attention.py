"""Binding of the attention layer's entry points (include/bi_model.h): the per-head norm with rotation
and softmax attention, forward and backward.  Argument checks and marshalling only."""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import _lib
from .api import _ptr, _raise_host, _stream


def _on(dev: torch.device):
    """The tensors' device made current for the call (nothing to do where it already is)."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, dev: torch.device, shape=None):
    # the library dereferences every pointer on the GPU: host memory must never reach it
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t: torch.Tensor, name: str, dev: torch.device, shape=None) -> int:
    """Elements between the tokens of a [T, heads, D] bf16 tensor whose heads are contiguous."""
    if t.get_device() == dev.index and t.dtype is torch.bfloat16 and t.dim() == 3 and shape in (None, t.shape):
        T, H, D = t.shape
        ld, sh, sd = t.stride()
        if T > 1 and sd == 1 and sh == D:  # what nearly every call has
            return ld
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {list(shape) if shape is not None else '[T, heads, D]'}, got {list(t.shape)}")
    T, H, D = t.shape
    ld, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous, strides are {t.stride()}")
    if T <= 1:
        return max(ld, H * D) if ld % 8 == 0 else -(-H * D // 8) * 8
    return ld


def _status(status: Optional[torch.Tensor], dev: torch.device) -> torch.Tensor:
    if status is None:
        return torch.empty(1, dtype=torch.int32, device=dev)
    _need(status, "status", torch.int32, dev)
    if status.numel() < 1:
        raise ValueError("status must hold one element")
    return status


def _qk_common(q, k, gq, gk, positions, inv_freq, dev):
    _rows(q, "q", dev)
    T, Hq, D = q.shape
    if k.dim() != 3 or k.shape[0] != T or k.shape[2] != D:
        raise ValueError(f"k must be [{T}, heads, {D}], got {list(k.shape)}")
    if (gq is None) != (gk is None):
        raise ValueError("gq and gk are given together or not at all")
    if gq is not None:
        _need(gq, "gq", torch.bfloat16, dev, (D,))
        _need(gk, "gk", torch.bfloat16, dev, (D,))
    _need(positions, "positions", torch.int32, dev, (T,))
    _need(inv_freq, "inv_freq", torch.float32, dev)
    return T, Hq, k.shape[1], D, 2 * inv_freq.numel()


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, gq: Optional[torch.Tensor], gk: Optional[torch.Tensor],
                 positions: torch.Tensor, inv_freq: torch.Tensor, eps: float, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """RMS norm of each head of q [T, Hq, D] and k [T, Hkv, D] with gains gq, gk [D] (None: no norm),
    then the rotation of its position: pairs (i, i + R/2), i < R/2 = len(inv_freq), turned by
    positions[t] * inv_freq[i]; elements past R pass (include/bi_model.h).  q and k may be slices of
    one projection's output.  Returns (q_out, k_out, status [1] i32)."""
    dev = q.device
    T, Hq, Hkv, D, R = _qk_common(q, k, gq, gk, positions, inv_freq, dev)
    q_ld, k_ld = _rows(q, "q", dev), _rows(k, "k", dev)
    if q_out is None:
        q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    if k_out is None:
        k_out = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev)
    qo_ld, ko_ld = _rows(q_out, "q_out", dev, q.shape), _rows(k_out, "k_out", dev, k.shape)
    st = _status(status, dev)
    with _on(dev):
        code = _lib.load().bi_qk_norm_rope(_ptr(q), _ptr(k), q_ld, k_ld, _ptr(gq), _ptr(gk), _ptr(positions),
                                           _ptr(inv_freq), float(eps), T, Hq, Hkv, D, R, _ptr(q_out), _ptr(k_out),
                                           qo_ld, ko_ld, _ptr(st), _stream(dev))
    _raise_host(code, "bi_qk_norm_rope")
    return q_out, k_out, st


def qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                     gq: Optional[torch.Tensor], gk: Optional[torch.Tensor], positions: torch.Tensor,
                     inv_freq: torch.Tensor, eps: float, dq: Optional[torch.Tensor] = None,
                     dk: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None):
    """The gradient of ``qk_norm_rope``.  Returns (dq, dk bf16, dgq, dgk [D] f32 or None, status)."""
    dev = q.device
    T, Hq, Hkv, D, R = _qk_common(q, k, gq, gk, positions, inv_freq, dev)
    q_ld, k_ld = _rows(q, "q", dev), _rows(k, "k", dev)
    gq_ld, gk_ld = _rows(dq_out, "dq_out", dev, q.shape), _rows(dk_out, "dk_out", dev, k.shape)
    lib = _lib.load()
    dgq = dgk = None
    if gq is not None:
        dgq, dgk = torch.empty(D, dtype=torch.float32, device=dev), torch.empty(D, dtype=torch.float32, device=dev)
        if ws is None:
            ws = torch.empty(max(lib.bi_qk_norm_rope_bwd_workspace_bytes(D), 256), dtype=torch.uint8, device=dev)
        _need(ws, "ws", torch.uint8, dev)
    if dq is None:
        dq = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    if dk is None:
        dk = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev)
    dq_ld, dk_ld = _rows(dq, "dq", dev, q.shape), _rows(dk, "dk", dev, k.shape)
    st = _status(status, dev)
    with _on(dev):
        code = lib.bi_qk_norm_rope_bwd(_ptr(dq_out), _ptr(dk_out), gq_ld, gk_ld, _ptr(q), _ptr(k), q_ld, k_ld, _ptr(gq),
                                       _ptr(gk), _ptr(positions), _ptr(inv_freq), float(eps), T, Hq, Hkv, D, R,
                                       _ptr(dq), _ptr(dk), dq_ld, dk_ld, _ptr(dgq), _ptr(dgk), _ptr(st), _ptr(ws),
                                       0 if ws is None else ws.numel(), _stream(dev))
    _raise_host(code, "bi_qk_norm_rope_bwd")
    return dq, dk, dgq, dgk, st


def _attn_common(q, k, v, q_offsets, k_offsets, k_lens, scale, dev):
    """(S, scale, k_offsets, q_ld, k_ld, v_ld) after the checks that forward and backward share."""
    q_ld, k_ld = _rows(q, "q", dev), _rows(k, "k", dev)
    v_ld = _rows(v, "v", dev, k.shape)
    if k.shape[2] != q.shape[2]:
        raise ValueError(f"q has heads of {q.shape[2]}, k of {k.shape[2]}")
    _need(q_offsets, "q_offsets", torch.int64, dev)
    S = q_offsets.numel() - 1
    if q_offsets.dim() != 1 or S < 0:
        raise ValueError("q_offsets must be [S + 1]")
    if k_offsets is None:
        if k.shape[0] != q.shape[0]:
            raise ValueError(f"k has {k.shape[0]} rows and q {q.shape[0]}: give k_offsets")
        k_offsets = q_offsets
    else:
        _need(k_offsets, "k_offsets", torch.int64, dev, q_offsets.shape)
    if k_lens is not None:
        _need(k_lens, "k_lens", torch.int32, dev, (S,))
    return S, float(q.shape[2] ** -0.5 if scale is None else scale), k_offsets, q_ld, k_ld, v_ld


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
             k_offsets: Optional[torch.Tensor] = None, k_lens: Optional[torch.Tensor] = None, causal: bool = True,
             scale: Optional[float] = None, ws: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """Softmax attention of q [Tq, Hq, D] over k, v [Tk, Hkv, D] (include/bi_model.h).  Sequence s has the
    query rows q_offsets[s]:q_offsets[s+1] and the key rows from k_offsets[s] on, k_lens[s] of them (all up
    to k_offsets[s+1] without k_lens); without k_offsets the keys are packed as the queries are.  Under
    ``causal`` the queries are the last positions of their sequence.  ``scale`` defaults to D ** -0.5.
    Rows in no sequence are left as they were.  Returns (out [Tq, Hq, D] bf16, lse [Hq, Tq] f32, status)."""
    dev = q.device
    S, scale, k_offsets, q_ld, k_ld, v_ld = _attn_common(q, k, v, q_offsets, k_offsets, k_lens, scale, dev)
    Tq, Hq, D = q.shape
    Tk, Hkv = k.shape[0], k.shape[1]
    lib = _lib.load()
    if ws is None:
        ws = torch.empty(max(lib.bi_attn_fwd_workspace_bytes(Tq, Tk, S, Hq, Hkv, D), 256), dtype=torch.uint8, device=dev)
    else:
        _need(ws, "ws", torch.uint8, dev)
    if out is None:
        out = torch.empty(Tq, Hq, D, dtype=torch.bfloat16, device=dev)
    else:
        _need(out, "out", torch.bfloat16, dev, q.shape)
    if lse is None:
        lse = torch.empty(Hq, Tq, dtype=torch.float32, device=dev)
    else:
        _need(lse, "lse", torch.float32, dev, (Hq, Tq))
    st = _status(status, dev)
    with _on(dev):
        code = lib.bi_attn_fwd(_ptr(q), _ptr(k), _ptr(v), q_ld, k_ld, v_ld, _ptr(q_offsets), _ptr(k_offsets),
                               _ptr(k_lens), S, Tq, Tk, Hq, Hkv, D, 1 if causal else 0, scale, _ptr(out), _ptr(lse),
                               _ptr(st), _ptr(ws), ws.numel(), _stream(dev))
    _raise_host(code, "bi_attn_fwd")
    return out, lse, st


def attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
             lse: torch.Tensor, q_offsets: torch.Tensor, k_offsets: Optional[torch.Tensor] = None,
             k_lens: Optional[torch.Tensor] = None, causal: bool = True, scale: Optional[float] = None,
             ws: Optional[torch.Tensor] = None, dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
             dv: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """The gradient of ``attn_fwd`` for dout [Tq, Hq, D], from its inputs and its results ``out`` and
    ``lse``.  dq, dk and dv may be slices of one buffer; rows in no sequence are left as they were.
    Returns (dq [Tq, Hq, D], dk, dv [Tk, Hkv, D] bf16, status)."""
    dev = q.device
    S, scale, k_offsets, q_ld, k_ld, v_ld = _attn_common(q, k, v, q_offsets, k_offsets, k_lens, scale, dev)
    Tq, Hq, D = q.shape
    Tk, Hkv = k.shape[0], k.shape[1]
    do_ld = _rows(dout, "dout", dev, q.shape)
    _need(out, "out", torch.bfloat16, dev, q.shape)
    _need(lse, "lse", torch.float32, dev, (Hq, Tq))
    lib = _lib.load()
    if ws is None:
        ws = torch.empty(max(lib.bi_attn_bwd_workspace_bytes(Tq, Tk, S, Hq, Hkv, D), 256), dtype=torch.uint8, device=dev)
    else:
        _need(ws, "ws", torch.uint8, dev)
    if dq is None:
        dq = torch.empty(Tq, Hq, D, dtype=torch.bfloat16, device=dev)
    if dk is None:
        dk = torch.empty(Tk, Hkv, D, dtype=torch.bfloat16, device=dev)
    if dv is None:
        dv = torch.empty(Tk, Hkv, D, dtype=torch.bfloat16, device=dev)
    dq_ld, dk_ld, dv_ld = (_rows(dq, "dq", dev, q.shape), _rows(dk, "dk", dev, k.shape), _rows(dv, "dv", dev, k.shape))
    st = _status(status, dev)
    with _on(dev):
        code = lib.bi_attn_bwd(_ptr(dout), do_ld, _ptr(q), _ptr(k), _ptr(v), q_ld, k_ld, v_ld, _ptr(out), _ptr(lse),
                               _ptr(q_offsets), _ptr(k_offsets), _ptr(k_lens), S, Tq, Tk, Hq, Hkv, D,
                               1 if causal else 0, scale, _ptr(dq), _ptr(dk), _ptr(dv), dq_ld, dk_ld, dv_ld, _ptr(st),
                               _ptr(ws), ws.numel(), _stream(dev))
    _raise_host(code, "bi_attn_bwd")
    return dq, dk, dv, st
