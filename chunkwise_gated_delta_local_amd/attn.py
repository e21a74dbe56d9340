"""Attention with a sliding window and a few first tokens that stay visible
(include/gdr_attn.h): the mixer that stands between layers of the gated delta
rule, for prompts, for single tokens over a cache of bounded size, and its
gradients.

As in ``api`` and ``mixer``, argument marshalling only. q, k and v may be slices
of a wider projection: the heads of a token are contiguous and the tokens evenly
strided (fewer than 2^22 elements apart; window_attn_step takes any stride).
"""
from __future__ import annotations

import ctypes
import math

import torch

from .api import _DTYPES, AttnProblem, load_library
from .mixer import _dense, _device, _grad_dtype, _launch, _out_dtype, _p, _seqs, _tokens, _workspace


def _attn(q, k, v, window, sinks, scale, N, out, grad=torch.float32, d_o=None):
    """Checks what the entry points share; q is [B, T, Nq, dk] or [N, Nq, dk]."""
    dev, io, lead = q.device, q.dtype, q.shape[:-2]
    if k.dim() != q.dim() or v.dim() != q.dim():
        raise ValueError("k and v must have as many axes as q")
    Nq, dk = q.shape[-2:]
    Nk, dv = v.shape[-2:]
    if Nq < 1 or Nk < 1 or dk < 1 or dv < 1:
        raise ValueError("heads and head dimensions must be positive")
    qs = _tokens(q, "q", q.shape, Nq * dk, io, dev)
    ks = _tokens(k, "k", lead + (Nk, dk), Nk * dk, io, dev)
    vs = _tokens(v, "v", lead + (Nk, dv), Nk * dv, io, dev)
    b, t = lead if len(lead) == 2 else (N, 1)
    t_io = _DTYPES[io]
    return AttnProblem(b, t, qs, ks, vs, N, Nq, Nk, dk, dv, window, sinks, dk ** -0.5 if scale is None else scale, t_io,
                       t_io if out is None else _DTYPES[out], t_io if d_o is None else _DTYPES[d_o.dtype], _DTYPES[grad])


def _check_window(window, sinks, scale):
    if not 1 <= window < 1 << 31 or not 0 <= sinks < (1 << 31) - window:
        raise ValueError("window must be positive, sinks >= 0 and their sum below 2^31")
    if scale is not None and not (scale > 0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")


def _caches(cache, lens, N, rows, k, v, dev, io):
    if len(cache) != 2:
        raise ValueError("cache must be (k_cache, v_cache)")
    _dense(cache[0], "k_cache", (N, rows) + k.shape[-2:], (io,), dev)
    _dense(cache[1], "v_cache", (N, rows) + v.shape[-2:], (io,), dev)
    if cache[0] is None or cache[1] is None:
        raise ValueError("cache must be (k_cache, v_cache)")
    _dense(lens, "lens", (N,), (torch.int32,), dev)


def window_attn_fwd(q, k, v, window, sinks=0, scale=None, cache=None, lens=None, cu_seqlens=None, cu_seqlens_cpu=None,
                    out_dtype=None):
    """Attention of each token to itself and the window - 1 tokens before it in
    its sequence, and to the sequence's first `sinks` tokens.

    q [B, T, Nq, dk], k [B, T, Nk, dk], v [B, T, Nk, dv], Nq a multiple of Nk,
    query head h reading key head h // (Nq / Nk), dk and dv at most 128; scale:
    dk ** -0.5 by default. cache: (k_cache [N, sinks + window, Nk, dk], v_cache
    [N, sinks + window, Nk, dv]) in the io dtype, read and then changed in place
    to hold the new tokens too; lens [N] int32: the tokens of each sequence
    before the call (None: none), read only. Without a cache the sequences begin
    here. Returns (o, lse), lse [B, T, Nq] float32 as window_attn_bwd takes it;
    out_dtype: dtype of o, the io dtype (default) or float32."""
    dev = _device(q)
    if q.dim() != 4:
        raise ValueError("expected q [B,T,Nq,dk]")
    _check_window(window, sinks, scale)
    out = _out_dtype(out_dtype, q.dtype)
    N, cu, host = _seqs(q.shape[0], cu_seqlens, cu_seqlens_cpu, dev)
    prob = _attn(q, k, v, window, sinks, scale, N, out)
    kc = vc = None
    if cache is not None:
        _caches(cache, lens, N, sinks + window, k, v, dev, q.dtype)
        kc, vc = cache
    elif lens is not None:
        raise ValueError("lens without a cache")
    o = torch.empty(q.shape[:3] + v.shape[3:], dtype=out, device=dev)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=dev)
    lib = load_library()
    ws, n = _workspace(lib.gdr_window_attn_fwd_workspace_size, prob, dev)
    _launch(lib.gdr_window_attn_fwd, dev, ctypes.byref(prob), _p(q), _p(k), _p(v), _p(kc), _p(vc), _p(lens), _p(cu),
            _p(host), _p(o), _p(lse), _p(ws), n)
    return o, lse


def window_attn_step(q, k, v, cache, lens, window, sinks=0, scale=None, out_dtype=None):
    """One token of each of N sequences: q [N, Nq, dk], k [N, Nk, dk], v [N, Nk,
    dv]; cache and lens as in window_attn_fwd. The token is written into the
    caches in place; the caller advances lens. A sequence with a negative lens is
    passed over: its caches stay, its output is zero. Returns o [N, Nq, dv]."""
    dev = _device(q)
    if q.dim() != 3:
        raise ValueError("expected q [N,Nq,dk]")
    _check_window(window, sinks, scale)
    out = _out_dtype(out_dtype, q.dtype)
    N = q.shape[0]
    prob = _attn(q, k, v, window, sinks, scale, N, out)
    if cache is None or lens is None:
        raise ValueError("cache and lens are required")
    _caches(cache, lens, N, sinks + window, k, v, dev, q.dtype)
    o = q.new_empty(q.shape[:2] + v.shape[2:], dtype=out)
    lib = load_library()
    ws, n = _workspace(lib.gdr_window_attn_step_workspace_size, prob, dev)
    _launch(lib.gdr_window_attn_step, dev, ctypes.byref(prob), _p(q), _p(k), _p(v), _p(cache[0]), _p(cache[1]), _p(lens),
            _p(o), _p(ws), n)
    return o


def window_attn_bwd(q, k, v, o, lse, d_o, window, sinks=0, scale=None, cu_seqlens=None, cu_seqlens_cpu=None,
                    grad_dtype=None):
    """Gradients of window_attn_fwd without a cache: dict dq, dk, dv (in
    grad_dtype: float32, the default, or the io dtype), given dL/do and the
    forward's o (each in the io dtype or float32) and lse."""
    dev = _device(q)
    if q.dim() != 4:
        raise ValueError("expected q [B,T,Nq,dk]")
    _check_window(window, sinks, scale)
    io, grad = q.dtype, _grad_dtype(grad_dtype, q.dtype)
    N, cu, host = _seqs(q.shape[0], cu_seqlens, cu_seqlens_cpu, dev)
    if o is None or lse is None or d_o is None:
        raise ValueError("o, lse and d_o are required")
    shape = q.shape[:3] + v.shape[3:]
    _dense(o, "o", shape, (io, torch.float32), dev)
    _dense(d_o, "d_o", shape, (io, torch.float32), dev)
    _dense(lse, "lse", q.shape[:3], (torch.float32,), dev)
    prob = _attn(q, k, v, window, sinks, scale, N, o.dtype, grad, d_o)
    dq, dk, dv = (torch.empty(x.shape, dtype=grad, device=dev) for x in (q, k, v))
    lib = load_library()
    ws, n = _workspace(lib.gdr_window_attn_bwd_workspace_size, prob, dev)
    _launch(lib.gdr_window_attn_bwd, dev, ctypes.byref(prob), _p(q), _p(k), _p(v), _p(o), _p(lse), _p(d_o), _p(cu),
            _p(host), _p(dq), _p(dk), _p(dv), _p(ws), n)
    return dict(dq=dq, dk=dk, dv=dv)
