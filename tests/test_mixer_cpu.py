"""What the layer operators refuse, found on the host before any device work."""
import ctypes

import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from chunkwise_gated_delta_local_amd import api

FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)
BIG = ctypes.c_size_t(1 << 46)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="passes placeholder addresses")


@pytest.fixture(scope="module")
def lib():
    return api.load_library()


def conv(**kw):
    d = dict(batch=2, seq_len=10, x_stride=64, num_seqs=2, channels=64, width=4, activation=1, io_dtype=1,
             param_dtype=0, dy_dtype=1, grad_dtype=0)
    d.update(kw)
    return api.ConvProblem(**d)


def scan(**kw):
    d = dict(batch=2, seq_len=10, x_stride=64, dt_stride=64, z_stride=64, b_stride=32, c_stride=32, num_seqs=2,
             channels=64, groups=2, state_dim=16, dt_softplus=1, io_dtype=1, out_dtype=1, dy_dtype=1, grad_dtype=0)
    d.update(kw)
    return api.ScanProblem(**d)


def norm(**kw):
    d = dict(rows=10, x_stride=64, cols=64, eps=1e-5, io_dtype=1, param_dtype=0, out_dtype=1, dy_dtype=1, grad_dtype=0)
    d.update(kw)
    return api.NormProblem(**d)


def size(lib, op, p):
    n = ctypes.c_size_t(0)
    return getattr(lib, "gdr_%s_workspace_size" % op)(ctypes.byref(p), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 2), (dict(seq_len=-1), 2), (dict(channels=0), 2), (dict(x_stride=63), 2), (dict(num_seqs=-1), 2),
    (dict(batch=1 << 20, seq_len=1 << 20), 2), (dict(io_dtype=2), 3), (dict(param_dtype=7), 3),
    (dict(io_dtype=0, param_dtype=1), 3), (dict(dy_dtype=9), 3), (dict(io_dtype=0, param_dtype=0, dy_dtype=0, grad_dtype=1), 3),
    (dict(width=1), 4), (dict(width=5), 4), (dict(activation=2), 4),
])
def test_conv_problems(lib, kw, code):
    assert size(lib, "conv_bwd", conv(**kw))[0] == code
    assert lib.gdr_last_error_message()


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 2), (dict(channels=0), 2), (dict(groups=3), 2), (dict(groups=0), 2), (dict(state_dim=0), 2),
    (dict(state_dim=65), 4), (dict(x_stride=1), 2), (dict(dt_stride=63), 2), (dict(b_stride=31), 2),
    (dict(c_stride=31), 2), (dict(io_dtype=5), 3), (dict(out_dtype=5), 3), (dict(io_dtype=0, out_dtype=1), 3),
    (dict(grad_dtype=4), 3), (dict(dt_softplus=2), 4), (dict(batch=1 << 16, seq_len=1 << 16), 2),
])
def test_scan_problems(lib, kw, code):
    assert size(lib, "scan_fwd", scan(**kw))[0] == code
    assert size(lib, "scan_bwd", scan(**kw))[0] == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 2), (dict(cols=0), 2), (dict(cols=16385, x_stride=16385), 4), (dict(x_stride=63), 2),
    (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(io_dtype=3), 3), (dict(param_dtype=3), 3),
    (dict(out_dtype=3), 3), (dict(io_dtype=0, param_dtype=1), 3),
])
def test_norm_problems(lib, kw, code):
    assert size(lib, "layer_norm_bwd", norm(**kw))[0] == code


def test_good_problems_and_their_workspaces(lib):
    assert size(lib, "conv_bwd", conv())[0] == 0
    assert size(lib, "scan_bwd", scan())[0] == 0 and size(lib, "scan_fwd", scan())[0] == 0
    assert size(lib, "layer_norm_bwd", norm())[0] == 0
    a, b = size(lib, "scan_bwd", scan(seq_len=100))[1], size(lib, "scan_bwd", scan(seq_len=10000))[1]
    assert 0 < a < b
    # a group's dB and dC once for each block of its channels, and the states before the tiles
    assert b >= 2 * 2 * 10000 * 32 * 4


def calls(lib):
    """name -> (function, arguments, index of every tensor argument, indices of the required ones)"""
    c, s, n = ctypes.byref(conv()), ctypes.byref(scan()), ctypes.byref(norm())
    s1, c1 = ctypes.byref(scan(seq_len=1)), ctypes.byref(conv(seq_len=1))
    F = FAKE
    return {
        "conv_fwd": (lib.gdr_conv_fwd, [c, F, F, F, F, None, None, F, F, None], (1, 2, 3, 4, 7, 8), (1, 2, 7)),
        "conv_step": (lib.gdr_conv_step, [c1, F, F, F, F, F, None], (1, 2, 3, 4, 5), (1, 2, 4, 5)),
        "conv_bwd": (lib.gdr_conv_bwd, [c, F, F, F, F, None, None, F, F, F, F, F, F, F, BIG, None],
                     (1, 2, 3, 4, 7, 8, 9, 10, 11, 12), (1, 2, 7, 9, 10)),
        "scan_fwd": (lib.gdr_scan_fwd, [s, F, F, F, F, F, F, F, F, F, None, None, F, F, None, ctypes.c_size_t(0), None],
                     (1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 13), (1, 2, 3, 4, 5, 12)),
        "scan_step": (lib.gdr_scan_step, [s1, F, F, F, F, F, F, F, F, F, F, None], tuple(range(1, 11)),
                      (1, 2, 3, 4, 5, 9, 10)),
        "scan_bwd": (lib.gdr_scan_bwd, [s, F, F, F, F, F, F, F, F, F, None, None, F, F, F, F, F, F, F, F, F, F, F, F,
                                        BIG, None],
                     tuple(range(1, 10)) + tuple(range(12, 23)), (1, 2, 3, 4, 5, 12, 14, 15, 16, 17, 18, 20)),
        "layer_norm_fwd": (lib.gdr_layer_norm_fwd, [n, F, F, F, F, F, F, None], (1, 2, 3, 4, 5, 6), (1, 4)),
        "layer_norm_bwd": (lib.gdr_layer_norm_bwd, [n, F, F, F, F, F, F, F, F, F, BIG, None],
                           tuple(range(1, 9)), (1, 2, 4, 5, 6)),
    }


NAMES = ("conv_fwd", "conv_step", "conv_bwd", "scan_fwd", "scan_step", "scan_bwd", "layer_norm_fwd", "layer_norm_bwd")


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
@pytest.mark.parametrize("name", ["conv_bwd", "scan_bwd", "layer_norm_bwd"])
def test_workspaces(lib, name):
    fn, args, _, _ = calls(lib)[name]
    at = len(args) - 3
    for ws, n in ((None, BIG), (ctypes.c_void_p((1 << 20) + 16), BIG), (FAKE, ctypes.c_size_t(16))):
        bad = list(args)
        bad[at], bad[at + 1] = ws, n
        assert fn(*bad) == 6


@no_gpu
@pytest.mark.parametrize("name,at", [("conv_fwd", 5), ("conv_bwd", 5), ("scan_fwd", 10), ("scan_bwd", 10)])
def test_sequence_offsets(lib, name, at):
    fn, args, _, _ = calls(lib)[name]
    one = dict(batch=1, num_seqs=2)
    p = conv(**one) if name.startswith("conv") else scan(**one)
    args[0] = ctypes.byref(p)
    assert fn(*args) == 2                                # num_seqs differs from batch
    for offs in ([1, 5, 10], [0, 6, 5], [0, 4, 9], [0, 4, 11]):
        t = torch.tensor(offs, dtype=torch.int32)
        bad = list(args)
        bad[at], bad[at + 1] = FAKE, ctypes.c_void_p(t.data_ptr())
        assert fn(*bad) == 5, offs
    bad = list(args)
    bad[at] = FAKE                                       # one copy alone
    assert fn(*bad) == 1
    t = torch.tensor([0, 5, 10], dtype=torch.int32)
    two = conv() if name.startswith("conv") else scan()
    bad = list(args)
    bad[0], bad[at], bad[at + 1] = ctypes.byref(two), FAKE, ctypes.c_void_p(t.data_ptr())
    assert fn(*bad) == 5                                 # packed sequences take one batch row


@no_gpu
def test_step_takes_one_token(lib):
    for name, p in (("conv_step", conv(seq_len=2)), ("scan_step", scan(seq_len=2)), ("conv_step", conv(batch=1, seq_len=1)),
                    ("scan_step", scan(batch=1, seq_len=1))):
        fn, args, _, _ = calls(lib)[name]
        assert fn(ctypes.byref(p), *args[1:]) == 2


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(1, 8, 64)
    for f in (lambda: gdr.conv_fwd(x, torch.zeros(64, 4)), lambda: gdr.conv_step(x[0], torch.zeros(8, 3, 64), torch.zeros(64, 4)),
              lambda: gdr.conv_bwd(x, torch.zeros(64, 4), x), lambda: gdr.scan_fwd(x, x, x, x, x),
              lambda: gdr.scan_step(x[0], x, x, x, x, x), lambda: gdr.scan_bwd(x, x, x, x, x, x),
              lambda: gdr.layer_norm_fwd(x), lambda: gdr.layer_norm_bwd(x, x, x, x)):
        with pytest.raises(ValueError):
            f()


def test_token_strides():
    """Slices of a wider projection give their stride; anything that is not evenly strided rows is refused."""
    from chunkwise_gated_delta_local_amd.mixer import _token_stride, _tokens
    wide = torch.zeros(3, 5, 40)
    assert _token_stride(wide[..., 8:16], "x", 8) == 40
    assert _token_stride(wide[..., 8:24].unflatten(-1, (2, 8)), "B", 16) == 40
    assert _token_stride(wide[:, 0, :8], "x", 8) == 200
    assert _token_stride(wide[:1, :1, :8], "x", 8) == 8 and _token_stride(wide[:, :1, :8], "x", 8) == 200
    assert _token_stride(wide[..., 3:4], "x", 1) == 40
    assert _tokens(wide, "x", wide.shape, 40, torch.float32, wide.device) == 40
    one = torch.zeros(1, 1, 8)
    for bad, width in ((wide[:, :4, :8], 8), (wide[..., ::2], 20), (one.expand(3, 5, 8), 8), (one.expand(1, 5, 8), 8),
                       (wide[0].t(), 5), (wide[:, 1:3, :8], 8), (torch.zeros(8).as_strided((4, 5), (1, 1)), 5),
                       (wide[..., :16].unflatten(-1, (2, 8))[..., :4], 8)):
        with pytest.raises(ValueError):
            _token_stride(bad, "x", width)
