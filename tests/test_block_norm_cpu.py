"""The gated RMS norm and the residual sum with its norms without a device: what they refuse before any device work, the
sizes of their launches, and that the bounds of their tests notice mistakes."""
import ctypes
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from chunkwise_gated_delta_local_amd import api
from mixer_common import U, f64, randn
from oracle import block_norm as ob
from test_launch_sizes_cpu import STAND_IN

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)
BIG = ctypes.c_size_t(1 << 46)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="passes placeholder addresses")


@pytest.fixture(scope="module")
def lib():
    return api.load_library()


def gated(**kw):
    d = dict(rows=10, x_stride=64, z_stride=64, cols=64, eps=1e-5, activation=1, io_dtype=1, param_dtype=0, out_dtype=1,
             dy_dtype=1, grad_dtype=0)
    d.update(kw)
    return api.GatedNormProblem(**d)


def residual(**kw):
    d = dict(rows=10, x_stride=64, residual_stride=64, gate_stride=64, cols=64, eps=1e-5, scale=1.0, gate=2, io_dtype=1,
             param_dtype=0, stream_dtype=0, out_dtype=1, dy_dtype=1, dh_dtype=0, grad_dtype=0, dres_dtype=0)
    d.update(kw)
    return api.ResidualNormProblem(**d)


def size(lib, op, p):
    n = ctypes.c_size_t(0)
    return getattr(lib, "gdr_%s_workspace_size" % op)(ctypes.byref(p), ctypes.byref(n)), n.value


def calls(lib, **kw):
    """name -> (function, arguments, index of every tensor argument, indices of the required ones)"""
    F = FAKE
    g = lambda: ctypes.byref(gated(**{k: v for k, v in kw.items() if k not in ("gate", "stream_dtype")}))
    r = lambda: ctypes.byref(residual(**{k: v for k, v in kw.items() if k != "activation"}))
    return {
        "gated_norm_fwd": (lib.gdr_gated_norm_fwd, [g(), F, F, F, F, F, None], (1, 2, 3, 4, 5), (1, 2, 4)),
        "gated_norm_bwd": (lib.gdr_gated_norm_bwd, [g(), F, F, F, F, F, F, F, F, F, BIG, None], tuple(range(1, 9)),
                           (1, 2, 3, 5, 6, 7)),
        "residual_norm_fwd": (lib.gdr_residual_norm_fwd, [r(), F, F, F, F, F, F, F, F, F, None], tuple(range(1, 10)),
                              (1, 2, 5, 6, 7)),
        "residual_norm_bwd": (lib.gdr_residual_norm_bwd, [r()] + [F] * 15 + [BIG, None], tuple(range(1, 15)),
                              (1, 2, 3, 7, 8, 9, 10, 11)),
    }


NAMES = ("gated_norm_fwd", "gated_norm_bwd", "residual_norm_fwd", "residual_norm_bwd")
SHARED = [(dict(rows=-1), 2), (dict(cols=0), 2), (dict(cols=16385, x_stride=16385), 4), (dict(x_stride=63), 2), (dict(eps=-1.0), 2),
          (dict(eps=float("nan")), 2), (dict(io_dtype=3), 3), (dict(param_dtype=3), 3), (dict(out_dtype=3), 3),
          (dict(io_dtype=0, param_dtype=1), 3), (dict(io_dtype=0, out_dtype=0, dy_dtype=1), 3), (dict(grad_dtype=2), 3)]


@pytest.mark.parametrize("kw,code", SHARED + [(dict(activation=0), 4), (dict(activation=3), 4), (dict(z_stride=63), 2)])
def test_gated_problems(lib, kw, code):
    assert size(lib, "gated_norm_bwd", gated(**kw))[0] == code
    assert lib.gdr_last_error_message()


@pytest.mark.parametrize("kw,code", SHARED + [(dict(scale=float("inf")), 2), (dict(scale=float("nan")), 2), (dict(gate=3), 4),
                                              (dict(gate=-1), 4), (dict(gate_stride=63), 2), (dict(residual_stride=63), 2),
                                              (dict(stream_dtype=4), 3), (dict(dh_dtype=4), 3), (dict(dres_dtype=4), 3),
                                              (dict(x_stride=(1 << 40) + 1), 2)])
def test_residual_problems(lib, kw, code):
    assert size(lib, "residual_norm_bwd", residual(**kw))[0] == code
    assert lib.gdr_last_error_message()


@no_gpu
@pytest.mark.parametrize("name", NAMES)
def test_pointers(lib, name):
    fn, args, tensors, required = calls(lib)[name]
    for i in tensors:
        bad = list(args)
        bad[i] = ODD
        assert fn(*bad) == 2, (name, i)
    for i in required:
        bad = list(args)
        bad[i] = None
        assert fn(*bad) == 1, (name, i)
    bad = list(args)
    bad[0] = None
    assert fn(*bad) == 1


@no_gpu
def test_gate_and_its_kind_agree(lib):
    for name, at in (("residual_norm_fwd", 5), ("residual_norm_bwd", 7)):
        fn, args, _, _ = calls(lib, gate=0)[name]
        assert fn(*args) == 1                            # a gate for GDR_GATE_NONE
        fn, args, _, _ = calls(lib, gate=1)[name]
        args[at] = None
        assert fn(*args) == 1
    fn, args, _, _ = calls(lib)["residual_norm_bwd"]
    args[9] = None                                       # a norm behind the block without its rstd
    assert fn(*args) == 1


@no_gpu
@pytest.mark.parametrize("name", ["gated_norm_bwd", "residual_norm_bwd"])
def test_workspaces(lib, name):
    fn, args, _, _ = calls(lib)[name]
    at = len(args) - 3
    for ws, n in ((None, BIG), (ctypes.c_void_p((1 << 20) + 16), BIG), (FAKE, ctypes.c_size_t(16))):
        bad = list(args)
        bad[at], bad[at + 1] = ws, n
        assert fn(*bad) == 6


def test_binding_refuses(monkeypatch):
    from chunkwise_gated_delta_local_amd import mixer as m
    x, r = torch.zeros(3, 8), torch.zeros(3)
    for f in (lambda: gdr.gated_norm_fwd(x, x), lambda: gdr.gated_norm_bwd(x, x, x, r), lambda: gdr.residual_norm_fwd(x, x),
              lambda: gdr.residual_norm_bwd(x, x, x, r)):
        with pytest.raises(ValueError):                  # tensors on the CPU
            f()
    monkeypatch.setattr(m, "_device", lambda t: t.device)
    monkeypatch.setattr(m, "_launch", lambda *a: pytest.fail("launched"))
    b = x.to(torch.bfloat16)
    bad = [lambda: m.gated_norm_fwd(x, x[:2]), lambda: m.gated_norm_fwd(x, b), lambda: m.gated_norm_fwd(x, x, activation="relu"),
           lambda: m.gated_norm_fwd(x, x, torch.zeros(7)), lambda: m.gated_norm_fwd(x, x, torch.zeros(8).half()),
           lambda: m.gated_norm_fwd(x, x, out_dtype=torch.float16), lambda: m.gated_norm_fwd(x[..., ::2], x[..., ::2]),
           lambda: m.gated_norm_fwd(x[:, :0], x[:, :0]), lambda: m.gated_norm_fwd(torch.zeros(()), torch.zeros(())),
           lambda: m.gated_norm_bwd(x, x, x[:2], r), lambda: m.gated_norm_bwd(x, x, x, r[:2]), lambda: m.gated_norm_bwd(x, x, x, r.double()),
           lambda: m.gated_norm_bwd(x, x, x.half(), r), lambda: m.gated_norm_bwd(x, x, x, r, grad_dtype=torch.float16),
           lambda: m.residual_norm_fwd(x, b), lambda: m.residual_norm_fwd(x, x[:2]), lambda: m.residual_norm_fwd(x, x, scale=float("nan")),
           lambda: m.residual_norm_fwd(b, x, torch.zeros(8), torch.zeros(8).to(torch.bfloat16)),
           lambda: m.residual_norm_fwd(b, x, torch.zeros(8), gate=torch.zeros(8).to(torch.bfloat16)),
           lambda: m.residual_norm_fwd(x, x, gate=torch.zeros(3)), lambda: m.residual_norm_fwd(b, x, gate=x),
           lambda: m.residual_norm_fwd(x, x, gate=x[:1].expand(3, 8)), lambda: m.residual_norm_fwd(x, x, torch.zeros(9)),
           lambda: m.residual_norm_bwd(x, x, x, r, x_weight=torch.zeros(8)), lambda: m.residual_norm_bwd(x, x, x, r, x_rstd=r),
           lambda: m.residual_norm_bwd(x, x[:2], x, r), lambda: m.residual_norm_bwd(x, x, x, r, d_h=x[:2]),
           lambda: m.residual_norm_bwd(x, x, x, r, d_h=x.double()), lambda: m.residual_norm_bwd(x, x, x, r[:2])]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            print("call %d was taken" % i)


CHILD = r"""
import ctypes, json, sys
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)           # before the library, so that its launches bind to it
sys.path[:0] = [sys.argv[2], sys.argv[2] + "/.."]
import test_block_norm_cpu as t
lib = t.api.load_library()
for name, kw in json.load(open(sys.argv[3])):
    fn, args, _, _ = t.calls(lib, **kw)[name]
    if name.endswith("bwd"):
        args[-2] = ctypes.c_size_t(t.size(lib, name, (t.gated if "gated" in name else t.residual)(**kw))[1])
    print("call", fn(*args), lib.gdr_last_error_message().decode(), flush=True)
"""


def test_launch_sizes(tmp_path):
    """Rows go round the grid, so that any number of them is taken; a workspace of the size that is asked for is enough."""
    (tmp_path / "stand_in.cpp").write_text(STAND_IN)
    so = str(tmp_path / "stand_in.so")
    subprocess.check_call(["g++", "-O1", "-shared", "-fPIC", str(tmp_path / "stand_in.cpp"), "-o", so])
    todo = []
    for io in (0, 1):
        for r, c in ((1, 1), (256, 4096), (1 << 21, 128), ((1 << 26) + 3, 5000), ((1 << 28) + 1, 1024), ((1 << 30) + 37, 2),
                     (1 << 38, 64), (1 << 40, 1), (1 << 40, 16384), (7, 513), (1 << 20, 8193)):
            kw = dict(rows=r, cols=c, x_stride=c, io_dtype=io, param_dtype=0, out_dtype=io, dy_dtype=io, grad_dtype=0)
            todo += [(name, dict(kw, z_stride=c)) for name in NAMES[:2]]
            todo += [(name, dict(kw, residual_stride=c, gate_stride=c)) for name in NAMES[2:]]
    (tmp_path / "todo.json").write_text(json.dumps(todo))
    out = subprocess.run([sys.executable, "-c", CHILD, so, HERE, str(tmp_path / "todo.json")], capture_output=True, text=True,
                         timeout=120)
    assert out.returncode == 0, out.stderr[-2000:]
    found, at = [], 0
    for line in out.stdout.splitlines():
        word = line.split()
        if word[0] == "launch":
            found.append(tuple(map(int, word[1:])))
            continue
        name, kw = todo[at]
        at += 1
        assert word[1] == "0" and found, (name, kw, line)
        for g, gyz, b, byz, lds in found:
            assert gyz == byz == 1 and 0 < b <= 1024 and 0 < g * b < 1 << 32 and lds <= 160 * 1024, (name, kw, found)
        found = []
    assert at == len(todo)


def test_bounds_notice_mistakes():
    """Mistakes planted in the formulas, seen from the bounds that the tests on the GPU use."""
    gen = torch.Generator().manual_seed(2)
    x, z, w = (f64(randn(gen, *s, dtype=torch.bfloat16)) for s in ((20, 130), (20, 130), (130,)))
    zm, C, half = np.abs(z).max(), 130, 2.0 ** -8
    far = lambda a, b, M, n: (np.abs(a - b) > 4 * (n * U * M + half * np.abs(b))).any()
    y, r = ob.gated_norm(x, z, w, "silu", 1e-5)
    assert far(ob.gated_norm(x[:, :-1], z[:, :-1], w[:-1], "silu", 1e-5)[0], y[:, :-1], np.abs(y[:, :-1]), C + 30 + 2 * zm)   # a column lost
    assert far(ob.gated_norm(x, z, w, "sigmoid", 1e-5)[0], y, np.abs(y), C + 30 + 2 * zm)
    assert far(ob.gated_norm(x, x, w, "silu", 1e-5)[0], y, np.abs(y), C + 30 + 2 * zm)
    dy = f64(randn(gen, 20, 130, dtype=torch.bfloat16))
    dx, dz, dw = ob.gated_norm_backward(x, z, dy, r, w, "silu")
    far32 = lambda a, b, M, n: (np.abs(a - b) > 4 * (n * U * M + 2.0 ** -24 * np.abs(b))).any()
    assert far32(ob.gated_norm_backward(x[:-1], z[:-1], dy[:-1], r[:-1], w, "silu")[2], dw, np.abs(dw) + 10, 60 + 2 * zm)     # a row lost
    hat = x * r[:, None]
    c = dy * ob.gate(z, "silu") * w
    M = r[:, None] * (np.abs(c) + np.abs(hat) * np.abs(c * hat).mean(-1, keepdims=True))
    assert far32(r[:, None] * c, dx, M, C + 60 + 4 * zm)                                                # without the mean
    assert far32(r[:, None] * (c - hat * (c * hat).sum(-1, keepdims=True) / 256), dx, M, C + 60 + 4 * zm)  # over padded columns
