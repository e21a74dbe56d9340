"""The operators that stand next to the gated delta rule in a layer
(include/gdr_mixer.h): the short causal convolution, the selective state space
scan, layer norm, the gated RMS norm, and the residual sum with its norms.

As in ``api``, argument marshalling only: torch supplies device memory and the
current HIP stream. Inputs that hold tokens ([B, T, ...]) may be slices of a
wider projection: the elements of a token are contiguous and the tokens evenly
strided (fewer than 2^22 elements apart in scan_fwd and scan_bwd). Everything
else is contiguous. Variable-length batches: B = 1 and
``cu_seqlens`` (with ``cu_seqlens_cpu``, its host copy, no device
synchronisation is needed); empty sequences are allowed.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .api import (_DTYPES, ConvProblem, GatedNormProblem, NormProblem, ResidualNormProblem, ScanProblem, _check,
                  load_library)

_ACTIVATIONS = {None: 0, "silu": 1}


def _device(t):
    if t.device.type != "cuda":
        raise ValueError("inputs must be on a GPU device")
    if t.dtype not in _DTYPES:
        raise ValueError("inputs must be bfloat16 or float32")
    return t.device


def _launch(fn, dev, *args):
    """Call a library entry point on the current stream of `dev`, with `dev` current."""
    stream = torch._C._cuda_getCurrentRawStream(dev.index)      # current_stream(dev).cuda_stream without its object
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _check(fn(*args, stream))
    _check(fn(*args, stream))


def _p(t):
    return None if t is None else t.data_ptr()


def _refuse(t, name, shape, dtypes):
    raise ValueError("%s must be %s in %s, on the inputs' device%s" % (
        name, list(shape), " or ".join(str(d) for d in dtypes),
        "" if t is None else " (got %s in %s on %s)" % (list(t.shape), t.dtype, t.device)))


def _dense(t, name, shape, dtypes, dev):
    """A contiguous tensor of this shape and one of these dtypes (None passes)."""
    if t is None:
        return
    if t.shape != shape or t.dtype not in dtypes or t.device != dev:
        _refuse(t, name, shape, dtypes)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _tokens(t, name, shape, width, dtype, dev):
    """The token stride (in elements) of an input [B, T, ...] or [N, ...] whose
    tokens hold `width` elements each."""
    if t.shape != shape or t.dtype != dtype or t.device != dev:
        _refuse(t, name, shape, (dtype,))
    return width if t.is_contiguous() else _token_stride(t, name, width)


def _token_stride(t, name, width):
    sizes, strides = list(t.shape), list(t.stride())
    inner = 1
    while inner < width:                        # the axes of a token
        n, st = sizes.pop(), strides.pop()
        if n > 1 and st != inner:
            raise ValueError("the elements of a token of %s must be contiguous" % name)
        inner *= n
    ld = rows = None
    for n, st in zip(reversed(sizes), reversed(strides)):
        if n == 1:
            continue
        if ld is None:
            ld, rows = st, n
        elif st == ld * rows:
            rows *= n
        else:
            raise ValueError("the tokens of %s must be evenly strided" % name)
    if ld is not None and ld < width:           # an expanded tensor, for one
        raise ValueError("the tokens of %s must not overlap" % name)
    return width if ld is None else ld


def _seqs(B, cu_seqlens, cu_seqlens_cpu, dev):
    """(number of sequences, device offsets, host offsets)"""
    if cu_seqlens is None:
        return B, None, None
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a vector of num_seqs + 1 offsets")
    host = (cu_seqlens if cu_seqlens_cpu is None else cu_seqlens_cpu).detach().to("cpu", torch.int32).contiguous()
    if host.shape != cu_seqlens.shape:
        raise ValueError("cu_seqlens and cu_seqlens_cpu must have the same length")
    return host.numel() - 1, cu_seqlens.detach().to(dev, torch.int32).contiguous(), host


def _grad_dtype(grad_dtype, io):
    if grad_dtype is None:
        return torch.float32
    if grad_dtype not in (io, torch.float32):
        raise ValueError("grad_dtype must be the io dtype or float32")
    return grad_dtype


def _workspace(size_fn, prob, dev):
    n = ctypes.c_size_t(0)
    _check(size_fn(ctypes.byref(prob), ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=dev) if n.value else None, n.value


# ---------------------------------------------------------------- short causal convolution
def _conv(x, weight, bias, activation, N, stride, grad=torch.float32, d_y=None):
    dev, io = x.device, x.dtype
    D = x.shape[-1]
    if weight.dim() != 2 or weight.shape[0] != D or weight.dtype not in (io, torch.float32):
        raise ValueError("weight must be [channels, width] in the io dtype or float32")
    _dense(weight, "weight", weight.shape, (weight.dtype,), dev)
    _dense(bias, "bias", (D,), (weight.dtype,), dev)
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be None or 'silu'")
    B, T = x.shape[:2] if x.dim() == 3 else (N, 1)
    return ConvProblem(B, T, stride, N, D, weight.shape[1], _ACTIVATIONS[activation], _DTYPES[io],
                       _DTYPES[weight.dtype], _DTYPES[io if d_y is None else d_y.dtype], _DTYPES[grad])


def conv_fwd(x, weight, bias=None, activation="silu", initial_state=None, output_final_state=True, cu_seqlens=None,
             cu_seqlens_cpu=None):
    """Short causal convolution over each sequence, one filter per channel.

    x [B, T, D]; weight [D, W] with W = 2, 3 or 4, bias [D] (io dtype or
    float32); activation "silu" or None. initial_state [N, W - 1, D] (io
    dtype): the inputs before the first token, oldest first; None: zeros.
    Returns (y, final_state or None); the final state is a later call's initial
    state."""
    dev = _device(x)
    if x.dim() != 3:
        raise ValueError("expected x [B,T,D]")
    stride = _tokens(x, "x", x.shape, x.shape[2], x.dtype, dev)
    N, cu, host = _seqs(x.shape[0], cu_seqlens, cu_seqlens_cpu, dev)
    prob = _conv(x, weight, bias, activation, N, stride)
    state = (N, weight.shape[1] - 1, x.shape[2])
    _dense(initial_state, "initial_state", state, (x.dtype,), dev)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    final = torch.empty(state, dtype=x.dtype, device=dev) if output_final_state else None
    _launch(load_library().gdr_conv_fwd, dev, ctypes.byref(prob), _p(x), _p(weight), _p(bias), _p(initial_state),
            _p(cu), _p(host), _p(y), _p(final))
    return y, final


def conv_step(x, state, weight, bias=None, activation="silu"):
    """One token of each of N sequences: x [N, D]; state [N, W - 1, D] is
    updated in place. Returns y [N, D]."""
    dev = _device(x)
    if x.dim() != 2:
        raise ValueError("expected x [N,D]")
    N, D = x.shape
    stride = _tokens(x, "x", x.shape, D, x.dtype, dev)
    prob = _conv(x, weight, bias, activation, N, stride)
    if state is None:
        raise ValueError("state is required")
    _dense(state, "state", (N, weight.shape[1] - 1, D), (x.dtype,), dev)
    y = x.new_empty((N, D))
    _launch(load_library().gdr_conv_step, dev, ctypes.byref(prob), _p(x), _p(weight), _p(bias), _p(state), _p(y))
    return y


def conv_bwd(x, weight, d_y, bias=None, activation="silu", initial_state=None, d_final_state=None, cu_seqlens=None,
             cu_seqlens_cpu=None, grad_dtype=None):
    """Gradients of conv_fwd: dict dx, dh0 (in grad_dtype: float32, the
    default, or the io dtype), dweight and dbias (float32), given dL/dy and
    dL/dfinal_state (None: zeros; both in the io dtype or float32)."""
    dev = _device(x)
    if x.dim() != 3:
        raise ValueError("expected x [B,T,D]")
    io, grad = x.dtype, _grad_dtype(grad_dtype, x.dtype)
    stride = _tokens(x, "x", x.shape, x.shape[2], io, dev)
    N, cu, host = _seqs(x.shape[0], cu_seqlens, cu_seqlens_cpu, dev)
    _dense(d_y, "d_y", x.shape, (io, torch.float32), dev)
    prob = _conv(x, weight, bias, activation, N, stride, grad, d_y)
    state = (N, weight.shape[1] - 1, x.shape[2])
    _dense(initial_state, "initial_state", state, (io,), dev)
    _dense(d_final_state, "d_final_state", state, (d_y.dtype,), dev)
    out = dict(dx=torch.empty(x.shape, dtype=grad, device=dev),
               dweight=torch.empty(weight.shape, dtype=torch.float32, device=dev),
               dbias=torch.empty(x.shape[2], dtype=torch.float32, device=dev),
               dh0=torch.empty(state, dtype=grad, device=dev))
    lib = load_library()
    ws, n = _workspace(lib.gdr_conv_bwd_workspace_size, prob, dev)
    _launch(lib.gdr_conv_bwd, dev, ctypes.byref(prob), _p(x), _p(weight), _p(bias), _p(initial_state), _p(cu),
            _p(host), _p(d_y), _p(d_final_state), _p(out["dx"]), _p(out["dweight"]), _p(out["dbias"]), _p(out["dh0"]),
            _p(ws), n)
    return out


# ---------------------------------------------------------------- selective state space scan
def _scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, N, out=None, grad=torch.float32, d_y=None):
    """Checks what the scan's entry points share; x is [B, T, D] or [N, D]."""
    dev, io, shape = x.device, x.dtype, x.shape
    ch, lead = shape[-1], shape[:-1]
    if A.dim() != 2:
        raise ValueError("A must be [channels, state] float32")
    if B.dim() != len(shape) + 1:
        raise ValueError("B and C must be [..., groups, state]")
    G, S = B.shape[-2:]
    f32 = (torch.float32,)
    _dense(A, "A", (ch, S), f32, dev)
    _dense(D, "D", (ch,), f32, dev)
    _dense(dt_bias, "dt_bias", (ch,), f32, dev)
    xs = _tokens(x, "x", shape, ch, io, dev)
    dts = _tokens(dt, "dt", shape, ch, io, dev)
    zs = 0 if z is None else _tokens(z, "z", shape, ch, io, dev)
    bs = _tokens(B, "B", lead + (G, S), G * S, io, dev)
    cs = _tokens(C, "C", lead + (G, S), G * S, io, dev)
    b, t = lead if len(lead) == 2 else (N, 1)
    t_io = _DTYPES[io]
    return ScanProblem(b, t, xs, dts, zs, bs, cs, N, ch, G, S, 1 if dt_softplus else 0, t_io,
                       t_io if out is None else _DTYPES[out], t_io if d_y is None else _DTYPES[d_y.dtype],
                       _DTYPES[grad], 0)


def _out_dtype(out_dtype, io):
    if out_dtype is None:
        return io
    if out_dtype not in (io, torch.float32):
        raise ValueError("out_dtype must be the io dtype or float32")
    return out_dtype


def scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False, initial_state=None,
             output_final_state=True, cu_seqlens=None, cu_seqlens_cpu=None, out_dtype=None):
    """Selective state space scan with a diagonal transition per channel.

        delta = dt + dt_bias (softplus of it with dt_softplus)
        h_t = exp(delta_t A) h_{t-1} + delta_t B_t x_t
        y_t = (sum over the state of C_t h_t + D x_t) silu(z_t)

    x, dt, z [B, T, D]; B, C [B, T, G, S], group g serving channels
    [g D / G, (g + 1) D / G); A [D, S] (negative: states decay), D and dt_bias
    [D] float32; states [N, D, S] float32, S at most 64. z, D, dt_bias and
    initial_state may be None. Returns (y, final_state or None); out_dtype: the
    io dtype (default) or float32."""
    dev = _device(x)
    if x.dim() != 3:
        raise ValueError("expected x [B,T,D]")
    out = _out_dtype(out_dtype, x.dtype)
    N, cu, host = _seqs(x.shape[0], cu_seqlens, cu_seqlens_cpu, dev)
    prob = _scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, N, out)
    state = (N, x.shape[2], B.shape[-1])
    _dense(initial_state, "initial_state", state, (torch.float32,), dev)
    y = torch.empty(x.shape, dtype=out, device=dev)
    final = torch.empty(state, dtype=torch.float32, device=dev) if output_final_state else None
    lib = load_library()
    ws, n = _workspace(lib.gdr_scan_fwd_workspace_size, prob, dev)
    _launch(lib.gdr_scan_fwd, dev, ctypes.byref(prob), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(z), _p(dt_bias),
            _p(initial_state), _p(cu), _p(host), _p(y), _p(final), _p(ws), n)
    return y, final


def scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=False, out_dtype=None):
    """One token of each of N sequences: x, dt, z [N, D]; B, C [N, G, S];
    state [N, D, S] float32 is updated in place. Returns y [N, D]."""
    dev = _device(x)
    if x.dim() != 2:
        raise ValueError("expected x [N,D]")
    out = _out_dtype(out_dtype, x.dtype)
    N = x.shape[0]
    prob = _scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, N, out)
    if state is None:
        raise ValueError("state is required")
    _dense(state, "state", (N, x.shape[1], B.shape[-1]), (torch.float32,), dev)
    y = x.new_empty(x.shape, dtype=out)
    _launch(load_library().gdr_scan_step, dev, ctypes.byref(prob), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(z),
            _p(dt_bias), _p(state), _p(y))
    return y


def scan_bwd(x, dt, A, B, C, d_y, D=None, z=None, dt_bias=None, dt_softplus=False, initial_state=None,
             d_final_state=None, cu_seqlens=None, cu_seqlens_cpu=None, grad_dtype=None):
    """Gradients of scan_fwd, given dL/dy (io dtype or float32) and
    dL/dfinal_state (float32, None: zeros): dict dx, ddt, dB, dC and, with z, dz
    (in grad_dtype: float32, the default, or the io dtype), dA, dD, ddt_bias
    and dh0 (float32). The states are formed again."""
    dev = _device(x)
    if x.dim() != 3:
        raise ValueError("expected x [B,T,D]")
    io, grad = x.dtype, _grad_dtype(grad_dtype, x.dtype)
    _dense(d_y, "d_y", x.shape, (io, torch.float32), dev)
    N, cu, host = _seqs(x.shape[0], cu_seqlens, cu_seqlens_cpu, dev)
    prob = _scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, N, None, grad, d_y)
    state = (N, x.shape[2], B.shape[-1])
    _dense(initial_state, "initial_state", state, (torch.float32,), dev)
    _dense(d_final_state, "d_final_state", state, (torch.float32,), dev)
    new = lambda shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=dev)
    out = dict(dx=new(x.shape, grad), ddt=new(x.shape, grad), dB=new(B.shape, grad), dC=new(C.shape, grad),
               dA=new(A.shape), dD=new(x.shape[2]), ddt_bias=new(x.shape[2]), dh0=new(state))
    if z is not None:
        out["dz"] = new(x.shape, grad)
    lib = load_library()
    ws, n = _workspace(lib.gdr_scan_bwd_workspace_size, prob, dev)
    _launch(lib.gdr_scan_bwd, dev, ctypes.byref(prob), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(z), _p(dt_bias),
            _p(initial_state), _p(cu), _p(host), _p(d_y), _p(d_final_state), _p(out["dx"]), _p(out["ddt"]),
            _p(out["dA"]), _p(out["dB"]), _p(out["dC"]), _p(out["dD"]), _p(out.get("dz")), _p(out["ddt_bias"]),
            _p(out["dh0"]), _p(ws), n)
    return out


# ---------------------------------------------------------------- layer norm
def _norm(x, weight, bias, eps, out, grad=torch.float32, d_y=None):
    dev, io = x.device, x.dtype
    if x.dim() < 1:
        raise ValueError("expected x [..., C]")
    C = x.shape[-1]
    if C < 1:
        raise ValueError("the last axis of x is empty")
    ld = C if x.is_contiguous() else _token_stride(x, "x", C)
    kinds = (io, torch.float32)
    _dense(weight, "weight", (C,), kinds, dev)
    _dense(bias, "bias", (C,), kinds if weight is None else (weight.dtype,), dev)
    param = io if weight is None and bias is None else (bias if weight is None else weight).dtype
    return NormProblem(x.numel() // C, ld, C, eps, _DTYPES[io], _DTYPES[param], _DTYPES[out],
                       _DTYPES[io if d_y is None else d_y.dtype], _DTYPES[grad], 0)


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out_dtype=None):
    """Layer norm over the last axis (at most 16384 elements) of x [..., C]:
    y = (x - mean) rstd weight + bias with rstd = 1 / sqrt(variance + eps);
    weight and bias [C] in the io dtype or float32. Returns (y, mean, rstd),
    mean and rstd [...] float32, as layer_norm_bwd takes them. out_dtype: the
    io dtype (default) or float32."""
    dev = _device(x)
    out = _out_dtype(out_dtype, x.dtype)
    prob = _norm(x, weight, bias, eps, out)
    y = x.new_empty(x.shape, dtype=out)
    mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
    rstd = torch.empty_like(mean)
    _launch(load_library().gdr_layer_norm_fwd, dev, ctypes.byref(prob), _p(x), _p(weight), _p(bias), _p(y), _p(mean),
            _p(rstd))
    return y, mean, rstd


def layer_norm_bwd(x, d_y, mean, rstd, weight=None, grad_dtype=None):
    """Gradients of layer_norm_fwd, given dL/dy (io dtype or float32) and the
    forward's mean and rstd: dict dx (in grad_dtype: float32, the default, or
    the io dtype), dweight and dbias (float32, summed over the rows)."""
    dev = _device(x)
    io, grad = x.dtype, _grad_dtype(grad_dtype, x.dtype)
    _dense(d_y, "d_y", x.shape, (io, torch.float32), dev)
    _dense(mean, "mean", x.shape[:-1], (torch.float32,), dev)
    _dense(rstd, "rstd", x.shape[:-1], (torch.float32,), dev)
    prob = _norm(x, weight, None, 0.0, io, grad, d_y)
    out = dict(dx=torch.empty(x.shape, dtype=grad, device=dev),
               dweight=torch.empty(x.shape[-1], dtype=torch.float32, device=dev),
               dbias=torch.empty(x.shape[-1], dtype=torch.float32, device=dev))
    lib = load_library()
    ws, n = _workspace(lib.gdr_layer_norm_bwd_workspace_size, prob, dev)
    _launch(lib.gdr_layer_norm_bwd, dev, ctypes.byref(prob), _p(x), _p(d_y), _p(weight), _p(mean), _p(rstd),
            _p(out["dx"]), _p(out["dweight"]), _p(out["dbias"]), _p(ws), n)
    return out


# ---------------------------------------------------------------- gated RMS norm
_GATES = {"silu": 1, "sigmoid": 2}


def _rows(t, name, shape, dtypes, dev):
    """The row stride of a tensor [..., C] of evenly strided rows."""
    if t.shape != shape or t.dtype not in dtypes or t.device != dev:
        _refuse(t, name, shape, dtypes)
    return shape[-1] if t.is_contiguous() else _token_stride(t, name, shape[-1])


def _cols(x):
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("expected x [..., C]")
    return x.shape[-1]


def _gated(x, z, weight, activation, eps, out, grad=torch.float32, d_y=None):
    dev, io, C = x.device, x.dtype, _cols(x)
    if activation not in _GATES:
        raise ValueError("activation must be 'silu' or 'sigmoid'")
    xs, zs = _rows(x, "x", x.shape, (io,), dev), _rows(z, "z", x.shape, (io,), dev)
    _dense(weight, "weight", (C,), (io, torch.float32), dev)
    t_io = _DTYPES[io]
    return GatedNormProblem(x.numel() // C, xs, zs, C, eps, _GATES[activation], t_io,
                            t_io if weight is None else _DTYPES[weight.dtype], _DTYPES[out],
                            t_io if d_y is None else _DTYPES[d_y.dtype], _DTYPES[grad])


def gated_norm_fwd(x, z, weight=None, activation="silu", eps=1e-5, out_dtype=None):
    """RMS norm over the last axis (at most 16384 elements) with a gate:
    y = x rstd weight act(z) with rstd = 1 / sqrt(mean(x^2) + eps) and act "silu"
    or "sigmoid". x, z [..., C] (rows evenly strided, slices of a projection for
    one); weight [C] in the io dtype or float32. Returns (y, rstd), rstd [...]
    float32 as gated_norm_bwd takes it. out_dtype: the io dtype (default) or
    float32."""
    dev = _device(x)
    out = _out_dtype(out_dtype, x.dtype)
    prob = _gated(x, z, weight, activation, eps, out)
    y = x.new_empty(x.shape, dtype=out)
    rstd = x.new_empty(x.shape[:-1], dtype=torch.float32)
    _launch(load_library().gdr_gated_norm_fwd, dev, ctypes.byref(prob), _p(x), _p(z), _p(weight), _p(y), _p(rstd))
    return y, rstd


def gated_norm_bwd(x, z, d_y, rstd, weight=None, activation="silu", grad_dtype=None):
    """Gradients of gated_norm_fwd, given dL/dy (io dtype or float32) and the
    forward's rstd: dict dx, dz (in grad_dtype: float32, the default, or the io
    dtype) and dweight (float32, summed over the rows)."""
    dev = _device(x)
    io, grad = x.dtype, _grad_dtype(grad_dtype, x.dtype)
    _dense(d_y, "d_y", x.shape, (io, torch.float32), dev)
    _dense(rstd, "rstd", x.shape[:-1], (torch.float32,), dev)
    prob = _gated(x, z, weight, activation, 0.0, io, grad, d_y)
    out = dict(dx=torch.empty(x.shape, dtype=grad, device=dev), dz=torch.empty(x.shape, dtype=grad, device=dev),
               dweight=torch.empty(x.shape[-1], dtype=torch.float32, device=dev))
    lib = load_library()
    ws, n = _workspace(lib.gdr_gated_norm_bwd_workspace_size, prob, dev)
    _launch(lib.gdr_gated_norm_bwd, dev, ctypes.byref(prob), _p(x), _p(z), _p(d_y), _p(weight), _p(rstd), _p(out["dx"]),
            _p(out["dz"]), _p(out["dweight"]), _p(ws), n)
    return out


# ---------------------------------------------------------------- residual sum with norms
def _residual(x, res, name, weight, x_weight, gate, scale, eps, out, grad=torch.float32, dres=torch.float32, d_y=None,
              d_h=None):
    dev, io, C = x.device, x.dtype, _cols(x)
    kinds, t_io = (io, torch.float32), _DTYPES[x.dtype]
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    xs, rs = _rows(x, "x", x.shape, (io,), dev), _rows(res, name, x.shape, kinds, dev)
    token = gate is not None and gate.dim() == x.dim() and (x.dim() > 1 or gate.dtype == io)
    param = next((t.dtype for t in (weight, x_weight, None if token else gate) if t is not None), io)
    if param not in kinds:
        raise ValueError("weight, x_weight and a gate per channel must be in the io dtype or float32")
    for t, label in ((weight, "weight"), (x_weight, "x_weight"), (None if token else gate, "gate")):
        _dense(t, label, (C,), (param,), dev)
    gs = _rows(gate, "gate", x.shape, (io,), dev) if token else 0
    return ResidualNormProblem(x.numel() // C, xs, rs, gs, C, eps, scale, 0 if gate is None else 2 if token else 1, t_io,
                               _DTYPES[param], _DTYPES[res.dtype], _DTYPES[out], t_io if d_y is None else _DTYPES[d_y.dtype],
                               t_io if d_h is None else _DTYPES[d_h.dtype], _DTYPES[grad], _DTYPES[dres])


def residual_norm_fwd(x, residual, weight=None, x_weight=None, gate=None, scale=1.0, eps=1e-5, out_dtype=None):
    """What lies between two blocks: h = residual + scale gate a, y = RMS norm of
    h times weight, where a is x, the block's output, or with x_weight the RMS
    norm of x times x_weight. All norms over the last axis (at most 16384).

    x [..., C]; residual [..., C] in the io dtype or float32 (rows evenly
    strided); gate: None, one a channel [C], or one a token, shaped like x in the
    io dtype; weight, x_weight and a channels' gate share a dtype, the io dtype or
    float32. Returns (y, h, rstd, x_rstd): y in out_dtype (the io dtype, or
    float32), h in residual's dtype, rstd and x_rstd (None without x_weight) [...]
    float32, as residual_norm_bwd takes them."""
    dev = _device(x)
    out = _out_dtype(out_dtype, x.dtype)
    prob = _residual(x, residual, "residual", weight, x_weight, gate, scale, eps, out)
    y = x.new_empty(x.shape, dtype=out)
    h = x.new_empty(x.shape, dtype=residual.dtype)
    rstd = x.new_empty(x.shape[:-1], dtype=torch.float32)
    x_rstd = None if x_weight is None else torch.empty_like(rstd)
    _launch(load_library().gdr_residual_norm_fwd, dev, ctypes.byref(prob), _p(x), _p(residual), _p(weight), _p(x_weight),
            _p(gate), _p(y), _p(h), _p(rstd), _p(x_rstd))
    return y, h, rstd, x_rstd


def residual_norm_bwd(x, h, d_y, rstd, weight=None, d_h=None, x_weight=None, x_rstd=None, gate=None, scale=1.0,
                      grad_dtype=None):
    """Gradients of residual_norm_fwd, given dL/dy and dL/dh (d_h, None: zeros;
    each in the io dtype or float32) and the forward's h, rstd and x_rstd: dict
    dx, dresidual, dweight and, with them, dx_weight and dgate (shaped like the
    gate). grad_dtype None (default): all float32; the io dtype: dx and a token
    gate's gradient in it, dresidual in h's dtype. Sums over rows are float32."""
    dev = _device(x)
    io, grad = x.dtype, _grad_dtype(grad_dtype, x.dtype)
    dres = torch.float32 if grad_dtype is None else h.dtype
    _dense(h, "h", x.shape, (io, torch.float32), dev)
    _dense(d_y, "d_y", x.shape, (io, torch.float32), dev)
    _dense(d_h, "d_h", x.shape, (io, torch.float32), dev)
    _dense(rstd, "rstd", x.shape[:-1], (torch.float32,), dev)
    _dense(x_rstd, "x_rstd", x.shape[:-1], (torch.float32,), dev)
    if (x_weight is None) != (x_rstd is None):
        raise ValueError("x_weight and x_rstd come together")
    prob = _residual(x, h, "h", weight, x_weight, gate, scale, 0.0, io, grad, dres, d_y, d_h)
    new = lambda shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=dev)
    C = x.shape[-1:]
    out = dict(dx=new(x.shape, grad), dresidual=new(x.shape, dres), dweight=new(C))
    if x_weight is not None:
        out["dx_weight"] = new(C)
    if gate is not None:
        out["dgate"] = new(x.shape, grad) if prob.gate == 2 else new(C)
    lib = load_library()
    ws, n = _workspace(lib.gdr_residual_norm_bwd_workspace_size, prob, dev)
    _launch(lib.gdr_residual_norm_bwd, dev, ctypes.byref(prob), _p(x), _p(h), _p(d_y), _p(d_h), _p(weight), _p(x_weight),
            _p(gate), _p(rstd), _p(x_rstd), _p(out["dx"]), _p(out["dresidual"]), _p(out["dweight"]),
            _p(out.get("dx_weight")), _p(out.get("dgate")), _p(ws), n)
    return out
