"""The layer operators on the GPU against oracle/mixer.py (float64), with the
bounds that tests/mixer_common.py derives."""
import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from mixer_common import T, U, close, f64, offsets, packed, randn, strided
from oracle import mixer as om

pytestmark = pytest.mark.gpu


def dev(t):
    return None if t is None else t.cuda()


# ---------------------------------------------------------------- convolution
def conv_case(dtype, lens, D, W, act=True, batch=False, state=True, bias=True, pad=0, param="f32", seed=0):
    gen = torch.Generator().manual_seed(seed)
    lead, cu = packed(lens, batch)
    N = len(lens)
    t, pt = T[dtype], T[param]
    c = dict(x=strided(randn(gen, *lead, D, dtype=t), pad), weight=randn(gen, D, W, dtype=pt, std=W ** -0.5),
             bias=randn(gen, D, dtype=pt, std=0.3) if bias else None,
             h0=randn(gen, N, W - 1, D, dtype=t) if state else None, d_y=randn(gen, *lead, D, dtype=t),
             dl=randn(gen, N, W - 1, D, dtype=t), cu=cu, lens=lens, act=act)
    n = int(sum(lens))
    c["ref"] = (f64(c["x"]).reshape(n, D), f64(c["weight"]), f64(c["bias"]) if bias else np.zeros(D),
                f64(c["h0"]) if state else np.zeros((N, W - 1, D)))
    return c


CONV = {
    "wide_packed": dict(dtype="bf16", lens=[1, 0, 200, 3, 129, 31], D=520, W=4),
    "wide_f32": dict(dtype="f32", lens=[130, 5, 0, 0, 1], D=516, W=3),
    "odd_channels": dict(dtype="bf16", lens=[40, 2, 0, 170], D=77, W=4),
    "odd_f32_no_state": dict(dtype="f32", lens=[33, 64], D=65, W=2, state=False, bias=False),
    "batch_strided": dict(dtype="bf16", lens=[150, 150], D=264, W=4, batch=True, pad=24),
    "strided_odd": dict(dtype="bf16", lens=[70], D=64, W=3, pad=5, param="bf16"),
    "seven_channels": dict(dtype="bf16", lens=[30, 0, 5], D=7, W=3, pad=2),
    "odd_and_long": dict(dtype="bf16", lens=[300, 301], D=523, W=4),
    "no_activation": dict(dtype="f32", lens=[10, 129], D=64, W=4, act=False),
    "shorter_than_taps": dict(dtype="bf16", lens=[1, 2, 1, 1, 2, 0, 1], D=64, W=4),
    "one_token": dict(dtype="f32", lens=[1], D=1, W=4),
}


def run_conv(c, back=False, **kw):
    a = dict(bias=dev(c["bias"]), activation="silu" if c["act"] else None, initial_state=dev(c["h0"]),
             cu_seqlens=dev(c["cu"]), cu_seqlens_cpu=c["cu"], **kw)
    if back:
        return gdr.conv_bwd(dev(c["x"]), dev(c["weight"]), dev(c["d_y"]), d_final_state=dev(c["dl"]), **a)
    return gdr.conv_fwd(dev(c["x"]), dev(c["weight"]), **a)


@pytest.mark.parametrize("case", sorted(CONV))
def test_conv_fwd(case):
    c = conv_case(**CONV[case])
    x, w, b, h0 = c["ref"]
    cu = offsets(c["lens"])
    y, last = run_conv(c)
    p, ref, rlast = om.conv(x, w, b, cu, h0, c["act"])
    Mp, _, _ = om.conv(np.abs(x), np.abs(w), np.abs(b), cu, np.abs(h0), False)
    # p is off by (W + 1) U Mp and |silu'| < 1.1; silu itself by 2 |p| + 8 of its value
    close(case + " y", y, ref, 1.1 * Mp + np.abs(ref), w.shape[1] + 1 + 2 * np.abs(p).max() + 8)
    assert np.array_equal(f64(last), rlast)


@pytest.mark.parametrize("grad", ["io", "f32"])
@pytest.mark.parametrize("case", sorted(CONV))
def test_conv_bwd(case, grad):
    c = conv_case(**CONV[case])
    x, w, b, h0 = c["ref"]
    cu, D = offsets(c["lens"]), x.shape[1]
    got = run_conv(c, back=True, grad_dtype=c["x"].dtype if grad == "io" else None)
    dy, dl = f64(c["d_y"]).reshape(x.shape), f64(c["dl"])
    p, _, _ = om.conv(x, w, b, cu, h0, c["act"])
    Mp, _, _ = om.conv(np.abs(x), np.abs(w), np.abs(b), cu, np.abs(h0), False)
    slope = om.silu_grad(p) if c["act"] else np.ones_like(p)
    ref = om.conv_backward(x, w, dy * slope, cu, h0, dl)
    # |silu''| <= 1/2 carries p's error; silu' has terms s and s (1 - s) |p| <= 1 each, of relative error 2 |p| + 8
    M = om.conv_backward(np.abs(x), np.abs(w), np.abs(dy) * (2.0 + Mp), cu, np.abs(h0), np.abs(dl))
    W = w.shape[1]
    for name, r, m, terms in zip(("dx", "dweight", "dbias", "dh0"), ref, M, (W + 1, len(x), len(x), W + 1)):
        close("%s %s" % (case, name), got[name], r, m, 2 * W + 2 * np.abs(p).max() + 12 + terms)
        assert got[name].dtype == (c["x"].dtype if grad == "io" and name in ("dx", "dh0") else torch.float32)


@pytest.mark.parametrize("dtype,D,W,pad", [("bf16", 512, 4, 0), ("f32", 100, 3, 0), ("bf16", 33, 2, 0), ("bf16", 64, 4, 8),
                                           ("f32", 530, 4, 3)])
def test_conv_step_continues_a_prompt(dtype, D, W, pad):
    """A prompt, then single tokens from its final state: bitwise the outputs of the whole."""
    c = conv_case(dtype, [9, 9, 9], D, W, batch=True, seed=3)
    y, last = run_conv(c)
    x, w, b = dev(c["x"]), dev(c["weight"]), dev(c["bias"])
    y0, state = gdr.conv_fwd(x[:, :6].contiguous(), w, b, initial_state=dev(c["h0"]))
    outs = [y0]
    for t in range(6, 9):
        xt = strided(x[:, t].contiguous()[None], pad)[0]
        outs.append(gdr.conv_step(xt, state, w, b)[:, None])
    assert torch.equal(torch.cat(outs, 1), y)
    assert torch.equal(state, last)


# ---------------------------------------------------------------- scan
def scan_case(dtype, lens, D, S, G=1, batch=False, state=True, gate=True, skip=True, bias=True, soft=True, pad=0,
              seed=0):
    gen = torch.Generator().manual_seed(seed)
    lead, cu = packed(lens, batch)
    N, t = len(lens), T[dtype]
    c = dict(x=strided(randn(gen, *lead, D, dtype=t), pad),
             dt=strided((randn(gen, *lead, D, std=0.5) if soft else torch.rand(*lead, D, generator=gen) * 0.3).to(t), pad),
             A=-torch.exp(randn(gen, D, S, std=0.5)), B=strided(randn(gen, *lead, G, S, dtype=t), pad),
             C=strided(randn(gen, *lead, G, S, dtype=t), pad), D=randn(gen, D) if skip else None,
             z=strided(randn(gen, *lead, D, dtype=t), pad) if gate else None,
             dt_bias=randn(gen, D, std=0.5, mean=-2.0 if soft else 0.05) if bias else None, soft=soft,
             h0=randn(gen, N, D, S) if state else None, d_y=randn(gen, *lead, D, dtype=t), dl=randn(gen, N, D, S),
             cu=cu, lens=lens)
    if not soft and bias:
        c["dt_bias"] = c["dt_bias"].abs()
    n = int(sum(lens))
    flat = lambda v, *s: f64(v).reshape(n, *s)
    pre = flat(c["dt"], D) + (f64(c["dt_bias"]) if bias else 0.0)
    delta = om.softplus(pre) if soft else pre
    c["ref"] = dict(x=flat(c["x"], D), delta=delta, A=f64(c["A"]), B=flat(c["B"], G, S), C=flat(c["C"], G, S),
                    skip=f64(c["D"]) if skip else np.zeros(D), cu=offsets(lens),
                    h0=f64(c["h0"]) if state else np.zeros((N, D, S)))
    c["abs"] = {k: np.abs(v) if k not in ("A", "cu") else v for k, v in c["ref"].items()}
    c["pre"], c["zf"] = pre, flat(c["z"], D) if gate else None
    # relative error of exp(delta A) along the longest sequence, and of delta
    eta = 2 * np.abs(pre).max() + 12 if soft else 1.0
    m = float(np.abs(delta[:, :, None] * c["ref"]["A"]).max()) if n else 0.0
    c["chain"], c["eta"] = max(lens) * (m * (20 + eta) + 3), eta
    return c


SCAN = {
    "one_piece": dict(dtype="f32", lens=[16], D=16, S=16),
    "packed": dict(dtype="bf16", lens=[1, 0, 129, 15, 128, 40, 0], D=40, S=16),
    "long": dict(dtype="f32", lens=[333], D=20, S=16),
    "batch_groups": dict(dtype="bf16", lens=[70, 70], D=72, S=16, G=3, batch=True),
    "state_1": dict(dtype="f32", lens=[37, 5], D=17, S=1),
    "state_7_odd": dict(dtype="bf16", lens=[130, 3], D=35, S=7, G=5),
    "state_24": dict(dtype="f32", lens=[90, 1, 17], D=36, S=24, G=2),
    "state_18_strided": dict(dtype="bf16", lens=[45, 45], D=34, S=18, G=2, batch=True, pad=6),
    "state_32": dict(dtype="bf16", lens=[140], D=33, S=32),
    "state_64": dict(dtype="f32", lens=[75, 2], D=18, S=64),
    "state_50": dict(dtype="bf16", lens=[41], D=16, S=50),
    "strided": dict(dtype="bf16", lens=[60, 60], D=48, S=16, batch=True, pad=3),
    "bare": dict(dtype="f32", lens=[50, 20], D=16, S=16, state=False, gate=False, skip=False, bias=False, soft=False),
    "no_gate": dict(dtype="bf16", lens=[50, 20], D=32, S=8, gate=False),
    "one_token": dict(dtype="f32", lens=[1], D=1, S=3),
    # few channels and long sequences: cut into segments that run side by side
    "segments": dict(dtype="f32", lens=[1500, 0, 300, 900], D=24, S=16),
    "segments_groups": dict(dtype="bf16", lens=[1100, 1100], D=20, S=24, G=2, batch=True),
    "segments_state_64": dict(dtype="bf16", lens=[2000], D=6, S=40, gate=False),
    "segments_bare": dict(dtype="f32", lens=[770, 769], D=3, S=5, state=False, gate=False, skip=False, bias=False,
                          soft=False),
    "many_short": dict(dtype="bf16", lens=[2, 1, 3, 0, 5, 1, 1, 2, 7, 4], D=50, S=16, G=2),
}


def scan_args(c):
    return [dev(c[k]) for k in ("x", "dt", "A", "B", "C")], dict(
        D=dev(c["D"]), z=dev(c["z"]), dt_bias=dev(c["dt_bias"]), dt_softplus=c["soft"])


def run_scan(c, back=False, **kw):
    a, k = scan_args(c)
    k.update(initial_state=dev(c["h0"]), cu_seqlens=dev(c["cu"]), cu_seqlens_cpu=c["cu"], **kw)
    if back:
        return gdr.scan_bwd(*a, dev(c["d_y"]), d_final_state=dev(c["dl"]), **k)
    return gdr.scan_fwd(*a, **k)


@pytest.mark.parametrize("out", ["io", "f32"])
@pytest.mark.parametrize("case", sorted(SCAN))
def test_scan_fwd(case, out):
    c = scan_case(**SCAN[case])
    y, last = run_scan(c, out_dtype=torch.float32 if out == "f32" else None)
    v, _, rlast = om.scan(**c["ref"])
    M, _, Mlast = om.scan(**c["abs"])
    kappa = c["chain"] + c["eta"] + c["ref"]["A"].shape[1] + 10
    close(case + " final state", last, rlast, Mlast, kappa)
    gate, kz = (1.0, 0.0) if c["zf"] is None else (om.silu(c["zf"]), 2 * np.abs(c["zf"]).max() + 10)
    close(case + " y", y, v * gate, M * np.abs(gate), kappa + kz)


@pytest.mark.parametrize("grad", ["io", "f32"])
@pytest.mark.parametrize("case", sorted(SCAN))
def test_scan_bwd(case, grad):
    c = scan_case(**SCAN[case])
    got = run_scan(c, back=True, grad_dtype=c["x"].dtype if grad == "io" else None)
    r, n = c["ref"], len(c["pre"])
    D, S = r["A"].shape
    dy, zf, dl = f64(c["d_y"]).reshape(n, D), c["zf"], f64(c["dl"])
    gate = np.ones_like(dy) if zf is None else om.silu(zf)
    ref = om.scan_backward(**r, ds=dy * gate, d_last=dl)
    M = om.scan_backward(**c["abs"], ds=np.abs(dy * gate), d_last=np.abs(dl), factor_A=np.abs(r["A"]))
    kz = 0.0 if zf is None else 2 * np.abs(zf).max() + 12
    # a product holds the chain of h and that of g; sums over states, channels of a group and tokens
    base = 2 * c["chain"] + 2 * c["eta"] + kz + S + 20
    ref, M = list(ref), list(M)
    if c["soft"]:                                # ddt = ddelta sigmoid(pre)
        s = 1 / (1 + np.exp(-c["pre"]))
        ref[1], M[1] = ref[1] * s, M[1] * s
        base += 2 * np.abs(c["pre"]).max() + 10
    for name, a, b, terms in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dh0"), ref, M, (0, 0, n, D, D, n, 0)):
        close("%s %s" % (case, name), got[name], a, b, base + terms)
        low = name in ("dx", "ddt", "dB", "dC") and grad == "io"
        assert got[name].dtype == (c["x"].dtype if low else torch.float32)
    close(case + " ddt_bias", got["ddt_bias"], ref[1].sum(0), M[1].sum(0), base + n)
    assert ("dz" in got) == (zf is not None)
    if zf is not None:
        v, _, _ = om.scan(**r)
        Mv, _, _ = om.scan(**c["abs"])
        s = 1 / (1 + np.exp(-zf))
        close(case + " dz", got["dz"], dy * v * om.silu_grad(zf), np.abs(dy) * Mv * s * (1 + np.abs(zf) * (1 - s)),
              base + kz)


@pytest.mark.parametrize("case,pad", [("batch_groups", 0), ("strided", 5)])
def test_scan_gradients_against_differences(case, pad):
    """Directional central differences of the GPU forward in fp32 itself."""
    c = scan_case("f32", [24, 24], 32, 16, G=2, batch=True, seed=11, pad=pad)
    a, k = scan_args(c)
    k["initial_state"] = dev(c["h0"])
    dy, dl = dev(c["d_y"]), dev(c["dl"])
    got = gdr.scan_bwd(*a, dy, d_final_state=dl, **k)
    gen = torch.Generator().manual_seed(5)
    slots = {"dx": (a, 0), "ddt": (a, 1), "dA": (a, 2), "dB": (a, 3), "dC": (a, 4), "dD": (k, "D"), "dz": (k, "z"),
             "ddt_bias": (k, "dt_bias"), "dh0": (k, "initial_state")}

    def loss():
        y, last = gdr.scan_fwd(*a, **k)
        return float((y.double() * dy.double()).sum() + (last.double() * dl.double()).sum())
    for name, (where, key) in slots.items():
        keep = where[key]
        d = torch.randn(keep.shape, generator=gen).cuda()
        d = d / d.norm() * keep.norm()
        eps = 2.0 ** -8
        where[key] = (keep + eps * d).contiguous()
        hi = loss()
        where[key] = (keep - eps * d).contiguous()
        lo = loss()
        where[key] = keep
        want, have = (hi - lo) / (2 * eps), float((got[name].double() * d.double()).sum())
        # third derivatives times eps^2 / 6 = 2.5e-6 and the rounding of the two sums (some 1e-6 of their terms' norm) / eps
        scale = float(got[name].double().norm() * d.double().norm())
        print(name, want, have, scale, flush=True)
        assert abs(want - have) <= 5e-3 * scale, (name, want, have)


@pytest.mark.parametrize("case", ["batch_groups", "strided", "state_24", "state_1", "state_64", "state_7_odd"])
def test_scan_step(case):
    """Every sequence's first token, from the initial state, in place."""
    kw = dict(SCAN[case])
    kw.update(lens=[1] * 5, batch=True)
    c = scan_case(**kw)
    a, k = scan_args(c)
    one = lambda t: None if t is None else t[:, 0]
    state = dev(c["h0"])
    y = gdr.scan_step(one(a[0]), one(a[1]), a[2], one(a[3]), one(a[4]), state, k["D"], one(k["z"]), k["dt_bias"],
                      k["dt_softplus"])
    v, _, rlast = om.scan(**c["ref"])
    M, _, Mlast = om.scan(**c["abs"])
    kappa = c["chain"] + c["eta"] + c["ref"]["A"].shape[1] + 10
    close(case + " state", state, rlast, Mlast, kappa)
    gate, kz = (1.0, 0.0) if c["zf"] is None else (om.silu(c["zf"]), 2 * np.abs(c["zf"]).max() + 10)
    close(case + " y", y, v * gate, M * np.abs(gate), kappa + kz)


# ---------------------------------------------------------------- layer norm
NORM = [("bf16", 3, 128), ("bf16", 1000, 128), ("bf16", 33, 8), ("bf16", 70, 512), ("bf16", 9, 1024), ("bf16", 7, 1032),
        ("bf16", 5, 4096), ("bf16", 3, 16384), ("bf16", 20, 7), ("bf16", 5, 1001), ("bf16", 2, 16383), ("f32", 600, 64),
        ("f32", 40, 100), ("f32", 6, 1), ("f32", 11, 1000), ("f32", 4, 2561), ("f32", 3, 8192), ("f32", 2, 16384),
        ("f32", 1, 4096), ("f32", 9, 513), ("f32", 2, 8191)]


def norm_case(dtype, R, C, pad=0, param="f32", weight=True):
    gen = torch.Generator().manual_seed(R * 7 + C)
    x = randn(gen, 1, R, C, dtype=T[dtype], std=1.5, mean=0.4)
    return (strided(x, pad)[0], randn(gen, C, dtype=T[param], mean=1.0, std=0.3) if weight else None,
            randn(gen, C, dtype=T[param]) if weight else None, randn(gen, R, C, dtype=T[dtype]))


def check_norm_fwd(name, x, w, b, y, mean, rstd, eps=1e-5):
    C = x.shape[-1]
    xf = f64(x)
    wf, bf = (np.ones(C), np.zeros(C)) if w is None else (f64(w), f64(b))
    ry, rm, rr = om.layer_norm(xf, wf, bf, eps)
    # a butterfly sum of C terms of sum |x|: fewer than 64 + 12 additions on any path
    e_m = 80 * np.abs(xf).mean(-1)
    close(name + " mean", mean, rm, e_m / 80, 80)
    # the variance carries 2 |x - mean| e_m / ... <= 2 e_m std, and 80 of its sum; rstd half of its relative error
    var = ((xf - rm[:, None]) ** 2).mean(-1) + eps
    k = 0.5 * (2 * e_m * np.sqrt(var) + 80 * var) / var + 6
    close(name + " rstd", rstd, rr, rr * k / k.max(), k.max())
    m = (np.abs((xf - rm[:, None]) * rr[:, None]) * (k[:, None] + 4) + (e_m * rr)[:, None]) * np.abs(wf) + 2 * np.abs(bf) + np.abs(ry)
    close(name + " y", y, ry, m, 1.0)


@pytest.mark.parametrize("dtype,R,C", NORM)
def test_layer_norm(dtype, R, C):
    x, w, b, dy = norm_case(dtype, R, C)
    y, mean, rstd = gdr.layer_norm_fwd(dev(x), dev(w), dev(b))
    check_norm_fwd("norm", x, w, b, y, mean, rstd)
    for grad in (None, x.dtype):
        got = gdr.layer_norm_bwd(dev(x), dev(dy), mean, rstd, dev(w), grad_dtype=grad)
        xf, d, mf, rf, wf = f64(x), f64(dy), f64(mean), f64(rstd), f64(w)
        dx, dw, db = om.layer_norm_backward(xf, d, mf, rf, wf)
        hat, c = np.abs(xf - mf[:, None]) * rf[:, None], np.abs(d * wf)
        M = rf[:, None] * (c + c.mean(-1, keepdims=True) + hat * (c * hat).mean(-1, keepdims=True))
        # a sum over a row: fewer than 76 additions on a path; over rows: at most R
        close("dx", got["dx"], dx, M, 100)
        close("dweight", got["dweight"], dw, (np.abs(d) * hat).sum(0), R + 10)
        close("dbias", got["dbias"], db, np.abs(d).sum(0), R + 10)


def test_layer_norm_forms():
    """No weights, a bf16 weight, strided rows, more leading axes, eps, fp32 output."""
    x, w, b, dy = norm_case("bf16", 12, 96, pad=5, param="bf16")
    y, mean, rstd = gdr.layer_norm_fwd(dev(x), dev(w), dev(b), eps=1e-3, out_dtype=torch.float32)
    check_norm_fwd("strided bf16 weight", x, w, b, y, mean, rstd, 1e-3)
    x3 = dev(x.contiguous()).view(3, 4, 96)
    y3, m3, r3 = gdr.layer_norm_fwd(x3)
    assert y3.shape == (3, 4, 96) and m3.shape == r3.shape == (3, 4)
    check_norm_fwd("plain", x, None, None, y3.view(12, 96), m3.view(-1), r3.view(-1))
    got = gdr.layer_norm_bwd(x3, dev(dy).view(3, 4, 96), m3, r3)
    dx, dw, db = om.layer_norm_backward(f64(x), f64(dy), f64(m3).reshape(-1), f64(r3).reshape(-1), np.ones(96))
    assert np.abs(f64(got["dx"]).reshape(12, 96) - dx).max() <= 100 * U * 20 * np.abs(f64(dy)).max()
    assert got["dx"].shape == (3, 4, 96) and got["dweight"].shape == (96,)
    const = torch.full((2, 64), 3.0, device="cuda")      # no variance: the bias alone
    y, mean, rstd = gdr.layer_norm_fwd(const, dev(w[:64].float().contiguous()), dev(b[:64].float().contiguous()))
    assert torch.equal(y, dev(b[:64].float()).expand(2, 64)) and torch.equal(mean, const[:, 0])


# ---------------------------------------------------------------- properties
def test_sequences_do_not_touch_each_other():
    """NaN and infinities in one sequence (its last and first tokens) leave the other outputs' bits."""
    for c, run in ((scan_case("bf16", [40, 130, 7], 32, 16), run_scan), (conv_case("bf16", [40, 130, 7], 64, 4), run_conv)):
        clean = run(c), run(c, back=True)
        for key in ("x", "dt", "B", "C", "z", "d_y"):
            if key in c:
                c[key][:, 40:43], c[key][:, 167:170] = float("nan"), float("inf")
        y, last = run(c)
        back = run(c, back=True)
        keep = torch.tensor(list(range(40)) + list(range(170, 177)), device="cuda")
        assert torch.equal(y[:, keep], clean[0][0][:, keep])
        assert torch.equal(last[[0, 2]], clean[0][1][[0, 2]])
        for k in ("dx", "ddt", "dz", "dB", "dC"):
            if k in back:
                assert torch.equal(back[k][:, keep], clean[1][k][:, keep]), k
        assert torch.equal(back["dh0"][[0, 2]], clean[1]["dh0"][[0, 2]])


@pytest.mark.parametrize("lens,D", [([70, 5, 0, 33], 32), ([3001], 16)])
def test_transitions_that_forget_at_once(lens, D):
    """exp(delta A) is 0 for A = -1e30 and for the lowest A, whose product with log2 e is no longer finite: the
    same bits. The lengths end inside a tile; the long sequence is cut into segments."""
    def all_of(low):
        c = scan_case("bf16", lens, D, 16)
        c["A"][1] = c["A"][:, 3] = low
        return [*run_scan(c), *run_scan(c, back=True).values()]
    for low in (-3e38, float("-inf")):
        for i, (a, b) in enumerate(zip(all_of(-1e30), all_of(low))):
            assert torch.isfinite(b).all() and torch.equal(a, b), (low, i)


def test_same_bits_again_and_on_another_stream():
    c, v = scan_case("bf16", [300, 41], 96, 16), conv_case("bf16", [300, 41], 96, 4)
    x, w, b, dy = (dev(t) for t in norm_case("bf16", 1000, 256))

    def all_of():
        y, m, r = gdr.layer_norm_fwd(x, w, b)
        out = [*run_scan(c), *run_scan(c, back=True).values(), *run_conv(v), *run_conv(v, back=True).values(), y, m, r]
        return out + list(gdr.layer_norm_bwd(x, dy, m, r, w).values())
    first = all_of()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = all_of()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, second))


def test_captured_and_replayed():
    """A captured step (convolution, scan, norm and their backward passes) gives the eager bits on every replay."""
    c, v = scan_case("bf16", [64, 64], 64, 16, batch=True), conv_case("bf16", [64, 64], 64, 4, batch=True)
    a, k = scan_args(c)
    xs = dev(v["x"])
    w, b, dy, h0, dl = (dev(v[n]) for n in ("weight", "bias", "d_y", "h0", "dl"))
    state, cstate = dev(c["h0"]).clone(), dev(v["h0"]).clone()

    def step():
        u, cl = gdr.conv_fwd(xs, w, b, initial_state=h0)
        y, last = gdr.scan_fwd(u, *a[1:], **k)
        o, m, r = gdr.layer_norm_fwd(y)
        g = gdr.layer_norm_bwd(y, dy, m, r, grad_dtype=y.dtype)
        gs = gdr.scan_bwd(u, *a[1:], g["dx"], grad_dtype=y.dtype, **k)
        gc = gdr.conv_bwd(xs, w, gs["dx"], b, initial_state=h0, d_final_state=dl, grad_dtype=y.dtype)
        t = gdr.conv_step(xs[:, 0], cstate, w, b)
        z = gdr.scan_step(t, a[1][:, 0], a[2], a[3][:, 0], a[4][:, 0], state, k["D"], None, k["dt_bias"], True)
        return [u, cl, y, last, o, *g.values(), *gs.values(), *gc.values(), t, z]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        xs.copy_(randn(torch.Generator().manual_seed(i), *xs.shape, dtype=xs.dtype).cuda())
        s0, c0 = state.clone(), cstate.clone()
        want = [t.clone() for t in step()]
        s1, c1 = state.clone(), cstate.clone()
        state.copy_(s0)
        cstate.copy_(c0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, out)), i
        assert torch.equal(state, s1) and torch.equal(cstate, c1), i


def test_outputs_stay_inside_their_rows():
    """Nothing is written behind the last token or sequence: the next allocation's bytes stay."""
    c = scan_case("bf16", [37, 5], 35, 7, G=5)
    a, k = scan_args(c)
    room = torch.full((4, 35, 7), 7.0, device="cuda")
    x2 = torch.cat([dev(c["x"])[0, :2], dev(c["x"])[0, :2]])[:2]
    gdr.scan_step(x2, a[1][0, :2], a[2], a[3][0, :2], a[4][0, :2], room[1:3], k["D"], None, k["dt_bias"], True)
    assert (room[0] == 7).all() and (room[3] == 7).all() and (room[1:3] != 7).any()
    rows = torch.full((4, 3, 33), 7.0, device="cuda", dtype=torch.bfloat16)
    v = conv_case("bf16", [2], 33, 4)
    gdr.conv_step(dev(v["x"])[0], rows[1:3], dev(v["weight"]), dev(v["bias"]))
    assert (rows[0] == 7).all() and (rows[3] == 7).all() and (rows[1:3, 2] != 7).any()


def test_more_than_the_caches_hold():
    """Calls of over 256 MB go past the caches: the bits of the same work in two smaller calls."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    x, dy, w, b = new(2, 11000, 4100), new(2, 11000, 4100), torch.randn(4100, 4, device="cuda"), torch.randn(4100, device="cuda")
    h0 = new(2, 3, 4100)
    y, last = gdr.conv_fwd(x, w, b, initial_state=h0)
    g = gdr.conv_bwd(x, w, dy, b, initial_state=h0, d_final_state=h0, grad_dtype=x.dtype)
    parts = [gdr.conv_bwd(x[i:i + 1], w, dy[i:i + 1], b, initial_state=h0[i:i + 1], d_final_state=h0[i:i + 1],
                          grad_dtype=x.dtype) for i in range(2)]
    for i in range(2):
        yi, li = gdr.conv_fwd(x[i:i + 1], w, b, initial_state=h0[i:i + 1])
        assert torch.equal(yi[0], y[i]) and torch.equal(li[0], last[i])
        assert torch.equal(parts[i]["dx"][0], g["dx"][i]) and torch.equal(parts[i]["dh0"][0], g["dh0"][i])
    # two orders of a sum of products: at most 160 additions on any path (runs of 128 tokens, their sums by 16
    # wavefronts), |silu'| < 1.1, and sum |dy u| <= |dy| |u|
    n_dy, n_u = (t.float().square().sum((0, 1)).sqrt().max() for t in (dy, x))
    for k, n in (("dweight", n_u + 10), ("dbias", 22000 ** 0.5)):
        assert float((g[k] - parts[0][k] - parts[1][k]).abs().max()) <= 2 * 160 * U * 1.1 * float(n_dy * n)
    N, D, S = 520, 4096, 16                              # states of 136 MB, read and written
    sx, sB = new(N, D), new(N, 1, S)
    A, st = -torch.rand(D, S, device="cuda"), torch.randn(N, D, S, device="cuda")
    st2 = st.clone()
    sy = gdr.scan_step(sx, sx, A, sB, sB, st, dt_softplus=True)
    for s in (slice(0, 260), slice(260, 520)):
        assert torch.equal(gdr.scan_step(sx[s], sx[s], A, sB[s], sB[s], st2[s], dt_softplus=True), sy[s])
    assert torch.equal(st, st2)
    x, dy = x.view(-1, 4100), dy.view(-1, 4100)
    y, m, r = gdr.layer_norm_fwd(x, b, b)
    g = gdr.layer_norm_bwd(x, dy, m, r, b, grad_dtype=x.dtype)
    for s in (slice(0, 9000), slice(9000, 22000)):
        ys, ms, rs = gdr.layer_norm_fwd(x[s], b, b)
        assert torch.equal(ys, y[s]) and torch.equal(ms, m[s]) and torch.equal(rs, r[s])
        assert torch.equal(gdr.layer_norm_bwd(x[s], dy[s], ms, rs, b, grad_dtype=x.dtype)["dx"], g["dx"][s])


def test_elements_past_31_bits():
    """Tensors of more than 2^31 elements: the sequence (or the rows) at their end against the same work alone, or
    against the definition where the split of the work differs. Every call is issued on more than 2^31 elements."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)
    n, D, S, tail = 131000, 16400, 4, 50
    x = new(1, n, D)
    cu = torch.tensor([0, n - tail, n], dtype=torch.int32)
    kw, end = dict(cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu), x[:, n - tail:].contiguous()
    w = torch.randn(D, 4, device="cuda") / 2
    y, last = gdr.conv_fwd(x, w, **kw)
    ye, le = gdr.conv_fwd(end, w)
    assert torch.equal(y[0, n - tail:], ye[0]) and torch.equal(last[1], le[0])
    del y
    dx = gdr.conv_bwd(x, w, x, grad_dtype=x.dtype, **kw)["dx"]
    assert torch.equal(dx[0, n - tail:], gdr.conv_bwd(end, w, end, grad_dtype=x.dtype)["dx"][0])
    del dx

    A, B = -torch.rand(D, S, device="cuda") - 0.1, new(1, n, 1, S)
    y, last = gdr.scan_fwd(x, x, A, B, B, z=x, dt_softplus=True, **kw)
    y = y[0, n - tail:].clone()
    g = gdr.scan_bwd(x, x, A, B, B, x, z=x, dt_softplus=True, grad_dtype=x.dtype, **kw)
    g = {k: (v[0, n - tail:] if v.dim() > 2 and k != "dh0" else v[1:] if k == "dh0" else v).clone() for k, v in g.items()}
    xf, Bf = f64(end[0]), f64(B[0, n - tail:])
    delta, gate, zm = om.softplus(xf), om.silu(xf), np.abs(xf).max()
    r = dict(x=xf, delta=delta, A=f64(A), B=Bf, C=Bf, skip=np.zeros(D), cu=offsets([tail]), h0=np.zeros((1, D, S)))
    a = {k: np.abs(v) if k not in ("A", "cu") else v for k, v in r.items()}
    eta = 2 * zm + 12
    chain = tail * (float((delta[:, :, None] * -r["A"]).max()) * (20 + eta) + 3)
    v, _, rlast = om.scan(**r)
    M, _, Mlast = om.scan(**a)
    close("final state", last[1:], rlast, Mlast, chain + eta + S + 10)
    close("y", y, v * gate, M * np.abs(gate), chain + eta + S + 20 + 2 * zm)
    ds, base = xf * gate, 2 * chain + 2 * eta + 2 * zm + 12 + S + 20
    zero = np.zeros((1, D, S))
    ref = om.scan_backward(**r, ds=ds, d_last=zero)
    M = om.scan_backward(**a, ds=np.abs(ds), d_last=zero, factor_A=-r["A"])
    for name, i, terms in (("dx", 0, 0), ("dB", 3, D), ("dC", 4, D), ("dh0", 6, 0)):
        close(name, g[name], ref[i], M[i], base + terms)
    s = 1 / (1 + np.exp(-xf))
    close("ddt", g["ddt"], ref[1] * s, M[1] * s, base + 2 * zm + 10)
    del y, g, x, B

    N, S = 8200, 16                                      # states of 2^31 elements
    sx, sB = new(N, D), new(N, 1, S)
    A, st = -torch.rand(D, S, device="cuda"), torch.full((N, D, S), 0.5, device="cuda")
    sy = gdr.scan_step(sx, sx, A, sB, sB, st, dt_softplus=True)
    st2 = torch.full((9, D, S), 0.5, device="cuda")
    ye = gdr.scan_step(sx[-9:], sx[-9:], A, sB[-9:], sB[-9:], st2, dt_softplus=True)
    assert torch.equal(sy[-9:], ye) and torch.equal(st[-9:], st2)
    del st

    x, w = new((1 << 24) + 70, 128), torch.randn(128, device="cuda")
    y, m, r = gdr.layer_norm_fwd(x, w, w)
    ys, ms, rs = gdr.layer_norm_fwd(x[-20000:], w, w)
    assert torch.equal(y[-20000:], ys) and torch.equal(m[-20000:], ms) and torch.equal(r[-20000:], rs)
    del y
    g = gdr.layer_norm_bwd(x, x, m, r, w, grad_dtype=x.dtype)
    assert torch.equal(g["dx"][-20000:], gdr.layer_norm_bwd(x[-20000:], x[-20000:], ms, rs, w, grad_dtype=x.dtype)["dx"])


def test_empty_calls():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    f = torch.float32
    w = z(64, 4, dtype=f) + 1
    h0, s0 = z(2, 3, 64) + 2, z(2, 64, 16, dtype=f) + 3
    y, last = gdr.conv_fwd(z(2, 0, 64), w, initial_state=h0)
    assert y.shape == (2, 0, 64) and torch.equal(last, h0)
    g = gdr.conv_bwd(z(2, 0, 64), w, z(2, 0, 64), initial_state=h0, d_final_state=h0)
    assert torch.equal(g["dh0"], h0.float()) and not g["dweight"].any() and not g["dbias"].any()
    A, B = z(64, 16, dtype=f) - 1, z(2, 0, 1, 16)
    y, last = gdr.scan_fwd(z(2, 0, 64), z(2, 0, 64), A, B, B, initial_state=s0)
    assert y.shape == (2, 0, 64) and torch.equal(last, s0)
    g = gdr.scan_bwd(z(2, 0, 64), z(2, 0, 64), A, B, B, z(2, 0, 64), initial_state=s0, d_final_state=s0)
    assert torch.equal(g["dh0"], s0) and not g["dA"].any() and not g["dD"].any() and not g["ddt_bias"].any()
    y, m, r = gdr.layer_norm_fwd(z(0, 64))
    g = gdr.layer_norm_bwd(z(0, 64), z(0, 64), m, r)
    assert y.shape == (0, 64) and not g["dweight"].any() and not g["dbias"].any()
    assert gdr.conv_step(z(0, 64), z(0, 3, 64), w).shape == (0, 64)
    assert gdr.scan_step(z(0, 64), z(0, 64), A, z(0, 1, 16), z(0, 1, 16), z(0, 64, 16, dtype=f)).shape == (0, 64)


def test_a_layer_of_them():
    """Convolution, gated delta rule and norm of every head, and convolution, scan and norm: a prompt in one call, and
    the same prompt cut in two with the states handed on."""
    gen = torch.Generator().manual_seed(1)
    B, n, H, d = 2, 96, 2, 64
    x = randn(gen, B, n, 3 * H * d, dtype=torch.bfloat16).cuda()
    w, wn = randn(gen, 3 * H * d, 4, std=0.5).cuda(), randn(gen, d, mean=1.0, std=0.1).cuda()
    beta = torch.sigmoid(randn(gen, B, n, H)).cuda()
    g = -torch.rand(B, n, H, generator=gen).cuda()

    def delta(x, beta, g, st):
        y, cst = gdr.conv_fwd(x, w, initial_state=st[0])
        q, k, v = (t.reshape(*t.shape[:2], H, d) for t in y.split(H * d, -1))
        k = torch.nn.functional.normalize(k.float(), dim=-1).to(k.dtype)
        o, S = gdr.chunk_fwd(q.contiguous(), k.contiguous(), v.contiguous(), beta.contiguous(), g=g.contiguous(),
                             initial_state=st[1])
        return gdr.layer_norm_fwd(o, wn)[0], (cst, S)
    whole, _ = delta(x, beta, g, (None, None))
    cut = lambda i, j: [t[:, i:j].contiguous() for t in (x, beta, g)]
    a, st = delta(*cut(0, 64), (None, None))
    b, _ = delta(*cut(64, n), st)
    assert torch.equal(torch.cat([a, b], 1), whole)      # cut at a chunk's end: the same arithmetic

    D, S = 128, 16
    wide = randn(gen, B, n, 2 * D + D + 2 * S, dtype=torch.bfloat16).cuda()
    cw, A = randn(gen, D, 4, std=0.5).cuda(), -torch.exp(randn(gen, D, S)).cuda()

    def selective(wide, st):
        xz, dt, BC = wide[..., :2 * D], wide[..., 2 * D:3 * D], wide[..., 3 * D:]
        u, cst = gdr.conv_fwd(xz[..., :D], cw, initial_state=st[0])
        Bm, Cm = (BC[..., i * S:(i + 1) * S].unflatten(-1, (1, S)) for i in (0, 1))
        y, h = gdr.scan_fwd(u, dt, A, Bm, Cm, z=xz[..., D:], dt_softplus=True, initial_state=st[1])
        return gdr.layer_norm_fwd(y)[0], (cst, h)
    whole, end = selective(wide, (None, None))
    a, st = selective(wide[:, :37].contiguous(), (None, None))
    outs = [a]
    for t in range(37, n):                               # single tokens from the prompt's states
        tok = wide[:, t]
        u = gdr.conv_step(tok[:, :D], st[0], cw)
        y = gdr.scan_step(u, tok[:, 2 * D:3 * D], A, tok[:, None, 3 * D:3 * D + S], tok[:, None, 3 * D + S:], st[1],
                          z=tok[:, D:2 * D], dt_softplus=True)
        outs.append(gdr.layer_norm_fwd(y)[0][:, None])
    assert torch.equal(st[0], end[0])
    # states: at most n tokens of relative error (|delta A| 40 + 3) U each; norms of bf16 outputs differ by their steps
    assert float((st[1] - end[1]).abs().max()) <= n * 400 * U * float(end[1].abs().max())
    diff = (torch.cat(outs, 1).float() - whole.float()).abs().max() / whole.float().abs().max()
    assert float(diff) <= 2 ** -6
