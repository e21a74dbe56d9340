"""The gated RMS norm and the residual sum with its norms on the GPU against oracle/block_norm.py (float64).

Bounds, in units of U = 2^-24 with C columns: rstd carries (C + 12) (a sum of C squares, half of it in the root, the
division); an element of a norm C + 20; act(z) and its slope 2 |z| + 12 of their terms, of which silu's slope has two
(s and z s (1 - s)). Sums over a row of c hat add C + 20 of the sum of absolute values, sums over rows their number."""
import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from mixer_common import T, close, f64, randn
from oracle import block_norm as ob

pytestmark = pytest.mark.gpu
EPS = 1e-5


def dev(t):
    return None if t is None else t.cuda()


def wide(t, pad):
    """The same values as a slice of wider rows."""
    if not pad:
        return t
    w = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype)
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


SHAPES = [(1, 1), (5, 3), (33, 128), (40, 127), (17, 64), (19, 65), (70, 129), (9, 256), (6, 513), (30, 1000), (4, 1025),
          (7, 2048), (5, 2561), (600, 4096), (3, 4097), (3, 8192), (3, 8200), (2, 16384), (3, 16001)]


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("dtype,param", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("R,C", SHAPES)
def test_gated_norm(R, C, dtype, param, act):
    gen = torch.Generator().manual_seed(R * 7 + C)
    t, pt = T[dtype], T[param]
    pad = (0, 8, 3)[C % 3]
    x, z, dy = wide(randn(gen, R, C, dtype=t, mean=0.3), pad), wide(randn(gen, R, C, dtype=t, std=2.0), pad), randn(gen, R, C, dtype=t)
    w = None if R == 17 else randn(gen, C, dtype=pt, mean=1.0, std=0.2)
    wf = np.ones(C) if w is None else f64(w)
    ref, r = ob.gated_norm(f64(x), f64(z), wf, act, EPS)
    zm = np.abs(f64(z)).max()
    for out in (None, torch.float32):
        y, rstd = gdr.gated_norm_fwd(dev(x), dev(z), dev(w), activation=act, eps=EPS, out_dtype=out)
        assert y.dtype == (t if out is None else out)
        close("y", y, ref, np.abs(ref), C + 30 + 2 * zm)
        close("rstd", rstd, r, np.abs(r), C + 12)
    r = f64(rstd)
    hat, dyf = np.abs(f64(x) * r[:, None]), np.abs(f64(dy))
    rx, rz, rw = ob.gated_norm_backward(f64(x), f64(z), f64(dy), r, wf, act)
    ga = np.abs(ob.gate(f64(z), act))
    s = ob.sigmoid(f64(z))
    slope = s + (np.abs(f64(z)) if act == "silu" else 1.0) * s * (1 - s)
    c = dyf * ga * np.abs(wf)
    Mx = r[:, None] * (c + hat * (c * hat).mean(-1, keepdims=True))
    for grad in (None, t):
        g = gdr.gated_norm_bwd(dev(x), dev(z), dev(dy), rstd, dev(w), activation=act, grad_dtype=grad)
        close("dx", g["dx"], rx, Mx, C + 60 + 4 * zm)
        close("dz", g["dz"], rz, dyf * hat * np.abs(wf) * slope, 60 + 4 * zm)
        close("dweight", g["dweight"], rw, (dyf * ga * hat).sum(0), R + 40 + 2 * zm)
        assert g["dx"].dtype == g["dz"].dtype == (grad or torch.float32) and g["dweight"].dtype == torch.float32
    if dtype == "bf16":                                   # an output gradient in fp32
        g = gdr.gated_norm_bwd(dev(x), dev(z), dev(dy).float(), rstd, dev(w), activation=act)
        close("dx", g["dx"], rx, Mx, C + 60 + 4 * zm)


def residual_case(R, C, dtype, stream, param, post, kind, weight=True, pad=0):
    gen = torch.Generator().manual_seed(R * 5 + C)
    t, st, pt = T[dtype], T[stream], T[param]
    c = dict(x=wide(randn(gen, R, C, dtype=t), pad), res=wide(randn(gen, R, C, dtype=st, std=2.0), pad),
             w=randn(gen, C, dtype=pt, mean=1.0, std=0.2) if weight else None,
             xw=randn(gen, C, dtype=pt, mean=1.0, std=0.2) if post else None,
             g={"none": None, "channel": randn(gen, C, dtype=pt, std=0.7),
                "token": wide(randn(gen, R, C, dtype=t, std=0.7), pad)}[kind])
    c["ref"] = dict(w=np.ones(C) if c["w"] is None else f64(c["w"]), xw=f64(c["xw"]),
                    g=np.ones(()) if c["g"] is None else f64(c["g"]), scale=0.6)
    return c


KINDS = [(dt, st, pa, post, kind) for dt, st, pa in (("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"), ("f32", "f32", "f32"))
         for post in (False, True) for kind in ("none", "channel", "token")]


@pytest.mark.parametrize("dtype,stream,param,post,kind", KINDS)
@pytest.mark.parametrize("R,C", SHAPES)
def test_residual_norm(R, C, dtype, stream, param, post, kind):
    c = residual_case(R, C, dtype, stream, param, post, kind, weight=R != 17, pad=(0, 8, 3)[R % 3])
    x, res, r = f64(c["x"]), f64(c["res"]), c["ref"]
    scale = float(np.float32(r["scale"]))
    r["scale"] = scale
    ry, rh, rr, rx = ob.residual_norm(x, res, r["w"], r["xw"], r["g"], scale, EPS)
    a = np.abs(x if rx is None else x * rx[:, None] * r["xw"])
    Mh = np.abs(res) + scale * np.abs(r["g"]) * a                # h is off by (C + 40) U Mh
    Ms = (Mh * np.abs(rh)).mean(-1) * rr ** 2                    # relative error of the mean square: twice that over it
    kw = dict(x_weight=dev(c["xw"]), gate=dev(c["g"]), scale=scale)
    for out in (None, torch.float32):
        y, h, rstd, x_rstd = gdr.residual_norm_fwd(dev(c["x"]), dev(c["res"]), dev(c["w"]), eps=EPS, out_dtype=out, **kw)
        assert y.dtype == (c["x"].dtype if out is None else out) and h.dtype == c["res"].dtype
        close("h", h, rh, Mh, C + 40)
        close("y", y, ry, (Mh + np.abs(rh) * (1 + 2 * Ms[:, None])) * rr[:, None] * np.abs(r["w"]), C + 60)
        close("rstd", rstd, rr, rr * (1 + 2 * Ms), C + 40)
        assert (x_rstd is None) == (not post)
        if post:
            close("x_rstd", x_rstd, rx, rx, C + 12)
    # backward, for h and the statistics as they came out
    gen = torch.Generator().manual_seed(1)
    dy, dh = randn(gen, R, C, dtype=c["x"].dtype), randn(gen, R, C, dtype=c["res"].dtype)
    for d_h, grad, f32 in ((dh, c["x"].dtype, False), (None, None, False), (dh.float(), None, True)):
        d_y = dy.float() * 1.001 if f32 else dy
        g = gdr.residual_norm_bwd(dev(c["x"]), h, dev(d_y), rstd, dev(c["w"]), d_h=dev(d_h), x_rstd=x_rstd, grad_dtype=grad, **kw)
        rs, xs = f64(rstd), f64(x_rstd)
        dyf, dhf = f64(d_y), np.zeros((R, C)) if d_h is None else f64(d_h)
        ref = ob.residual_norm_backward(x, f64(h), dyf, dhf, rs, xs, r["w"], r["xw"], r["g"], scale)
        hat = np.abs(f64(h) * rs[:, None])
        e = np.abs(dyf * r["w"])
        Md = np.abs(dhf) + rs[:, None] * (e + hat * (e * hat).mean(-1, keepdims=True))
        m = scale * np.abs(r["g"]) * Md
        if post:
            xh = np.abs(x * xs[:, None])
            Mx = xs[:, None] * (m * np.abs(r["xw"]) + xh * (m * np.abs(r["xw"]) * xh).mean(-1, keepdims=True))
            Ma = xh * np.abs(r["xw"])
        else:
            Mx, Ma = m, np.abs(x)
        close("dresidual", g["dresidual"], ref["dresidual"], Md, C + 60)
        close("dx", g["dx"], ref["dx"], Mx, 2 * C + 120)
        close("dweight", g["dweight"], ref["dweight"], (np.abs(dyf) * hat).sum(0), R + 30)
        assert g["dx"].dtype == (grad or torch.float32) and g["dresidual"].dtype == (torch.float32 if grad is None else h.dtype)
        if post:
            close("dx_weight", g["dx_weight"], ref["dx_weight"], (m * xh).sum(0), R + C + 90)
        if kind == "token":
            close("dgate", g["dgate"], ref["dgate"], scale * Md * Ma, C + 90)
        elif kind == "channel":
            close("dgate", g["dgate"], ref["dgate"].sum(0), (scale * Md * Ma).sum(0), R + C + 90)
        assert ("dgate" in g) == (kind != "none") and ("dx_weight" in g) == post


@pytest.mark.parametrize("post,kind", [(False, "none"), (False, "token"), (True, "none"), (True, "channel")])
@pytest.mark.parametrize("C", [8, 24, 56, 60, 72, 100, 112, 120, 136, 224, 232, 264, 448, 456, 520, 768, 896, 904, 1023, 1024, 12000])
def test_widths_beside_a_stream_in_fp32(C, post, kind):
    """Rows that are moved in pieces of four and of eight elements."""
    test_residual_norm(21, C, "bf16", "f32", "bf16", post, kind)


def test_axes_and_vectors():
    """Any number of leading axes; x of one axis is one row, with a gate in another dtype than its own a channel's."""
    gen = torch.Generator().manual_seed(3)
    x, z, w = randn(gen, 2, 3, 4, 32).cuda(), randn(gen, 2, 3, 4, 32).cuda(), randn(gen, 32).cuda()
    y, r = gdr.gated_norm_fwd(x, z, w)
    y2, r2 = gdr.gated_norm_fwd(x.reshape(24, 32), z.reshape(24, 32), w)
    assert torch.equal(y.reshape(24, 32), y2) and torch.equal(r.reshape(24), r2) and r.shape == (2, 3, 4)
    a = gdr.residual_norm_fwd(x, z, w, gate=x)
    b = gdr.residual_norm_fwd(x.reshape(24, 32), z.reshape(24, 32), w, gate=x.reshape(24, 32))
    assert torch.equal(a[0].reshape(24, 32), b[0]) and torch.equal(a[1].reshape(24, 32), b[1])
    row = x[0, 0, 0]
    assert torch.equal(gdr.residual_norm_fwd(row, row, gate=w)[1], gdr.residual_norm_fwd(row[None], row[None], gate=w)[1][0])


def test_same_bits_and_rows_alone():
    gen = torch.Generator().manual_seed(4)
    x, z = (randn(gen, 3000, 128, dtype=torch.bfloat16).cuda() for _ in range(2))
    w = randn(gen, 128).cuda()
    y, r = gdr.gated_norm_fwd(x, z, w)
    g = gdr.gated_norm_bwd(x, z, x, r, w)
    a = gdr.residual_norm_fwd(x, z, w, x_weight=w, gate=z)
    d = gdr.residual_norm_bwd(x, a[1], x, a[2], w, d_h=z, x_weight=w, x_rstd=a[3], gate=z)
    for _ in range(2):
        assert all(torch.equal(g[k], v) for k, v in gdr.gated_norm_bwd(x, z, x, r, w).items())
        again = gdr.residual_norm_bwd(x, a[1], x, a[2], w, d_h=z, x_weight=w, x_rstd=a[3], gate=z)
        assert all(torch.equal(d[k], v) for k, v in again.items())
    s = slice(1000, 1017)
    assert torch.equal(gdr.gated_norm_fwd(x[s], z[s], w)[0], y[s])
    assert torch.equal(gdr.gated_norm_bwd(x[s], z[s], x[s], r[s], w)["dx"], g["dx"][s])
    assert torch.equal(gdr.residual_norm_fwd(x[s], z[s], w, x_weight=w, gate=z[s])[0], a[0][s])


def test_rows_do_not_touch():
    """NaN and Inf in a row stay in it (sums over rows excepted)."""
    gen = torch.Generator().manual_seed(5)
    for C in (64, 1000, 5000):
        x, z = (randn(gen, 50, C, dtype=torch.bfloat16).cuda() for _ in range(2))
        base, r = gdr.gated_norm_fwd(x, z)
        rb = gdr.residual_norm_fwd(x, z)
        bad = x.clone()
        bad[7, 3], bad[9, 0] = float("nan"), float("inf")
        keep = torch.ones(50, dtype=torch.bool, device="cuda")
        keep[7] = keep[9] = False
        y, _ = gdr.gated_norm_fwd(bad, z)
        h = gdr.residual_norm_fwd(bad, z)
        assert torch.equal(y[keep], base[keep]) and torch.isnan(y[7]).all()
        assert torch.equal(h[0][keep], rb[0][keep]) and torch.isnan(h[0][7]).all()


def test_gates_at_their_ends():
    """z of 200, -200 and infinities: silu and sigmoid go to their limits, forward and backward."""
    z = torch.tensor([[200.0, -200.0, 90.0, -90.0, float("inf"), 0.0]]).cuda()
    x, dy = torch.ones_like(z), torch.ones_like(z)
    y, r = gdr.gated_norm_fwd(x, z, activation="sigmoid", eps=0.0)
    assert y[0, 0] == 1 and y[0, 1] == 0 and y[0, 4] == 1 and y[0, 5] == 0.5
    y, _ = gdr.gated_norm_fwd(x, z[:, :4].repeat(1, 2)[:, :6], eps=0.0)
    assert y[0, 0] == 200 and abs(float(y[0, 1])) < 1e-30
    for act in ("silu", "sigmoid"):
        g = gdr.gated_norm_bwd(x, z[:, [0, 1, 2, 3, 5, 5]], dy, r, activation=act)
        assert all(torch.isfinite(v).all() for v in g.values())


def test_graph_and_stream():
    gen = torch.Generator().manual_seed(6)
    x, z, w = randn(gen, 300, 512).cuda(), randn(gen, 300, 512).cuda(), randn(gen, 512).cuda()

    def all_of_it():
        y, r = gdr.gated_norm_fwd(x, z, w)
        a = gdr.residual_norm_fwd(y, z, w, x_weight=w, gate=w)
        d = gdr.residual_norm_bwd(y, a[1], x, a[2], w, d_h=z, x_weight=w, x_rstd=a[3], gate=w)
        g = gdr.gated_norm_bwd(x, z, d["dx"], r, w)
        return [y, a[0], a[1], *d.values(), *g.values()]
    want = all_of_it()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = all_of_it()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = all_of_it()
    for i in range(3):
        x.copy_(randn(gen, 300, 512))
        graph.replay()
        want = all_of_it()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
        torch.cuda.synchronize()


def test_gradients_against_differences():
    """Along random directions, in fp32 with steps of 1e-2: a difference carries the forward's 1e-6 of y twice over the
    step, and the third derivative times its square."""
    gen = torch.Generator().manual_seed(7)
    R, C = 6, 96
    x, z, dy, dh = (randn(gen, R, C).cuda() for _ in range(4))
    w, xw, g = (randn(gen, C, mean=1.0, std=0.2).cuda() for _ in range(3))
    step = lambda t: randn(gen, *t.shape).cuda()

    def slope(f, t, s=1e-2):
        d = step(t)
        return float((f(t + s * d) - f(t - s * d)) / (2 * s)), d
    r = gdr.gated_norm_fwd(x, z, w)[1]
    got = gdr.gated_norm_bwd(x, z, dy, r, w)
    for name, t, f in (("dx", x, lambda t: gdr.gated_norm_fwd(t, z, w)[0]), ("dz", z, lambda t: gdr.gated_norm_fwd(x, t, w)[0]),
                       ("dweight", w, lambda t: gdr.gated_norm_fwd(x, z, t)[0])):
        s, d = slope(lambda t: (f(t).double() * dy.double()).sum(), t)
        assert abs(s - float((got[name].double() * d.double()).sum())) <= 5e-3 * float(got[name].norm()) * C ** 0.5 / 5, name
    fwd = lambda x=x, z=z, w=w, xw=xw, g=g: gdr.residual_norm_fwd(x, z, w, x_weight=xw, gate=g, scale=0.7)
    _, h, r, xr = fwd()
    got = gdr.residual_norm_bwd(x, h, dy, r, w, d_h=dh, x_weight=xw, x_rstd=xr, gate=g, scale=0.7)
    for name, key, t in (("dx", "x", x), ("dresidual", "z", z), ("dweight", "w", w), ("dx_weight", "xw", xw), ("dgate", "g", g)):
        def f(t):
            y, h, _, _ = fwd(**{key: t})
            return (y.double() * dy.double()).sum() + (h.double() * dh.double()).sum()
        s, d = slope(f, t)
        assert abs(s - float((got[name].double() * d.double()).sum())) <= 5e-3 * float(got[name].norm()) * C ** 0.5 / 5, name


def test_many_rows():
    """More than 2^31 elements: rows at the end against the same rows alone."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((1 << 24) + 70, 128, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(128, device="cuda")
    y, r = gdr.gated_norm_fwd(x, x, w)
    s = slice(-5000, None)
    ys, rs = gdr.gated_norm_fwd(x[s], x[s], w)
    assert torch.equal(y[s], ys) and torch.equal(r[s], rs)
    del y
    g = gdr.gated_norm_bwd(x, x, x, r, w, grad_dtype=x.dtype)
    gs = gdr.gated_norm_bwd(x[s], x[s], x[s], rs, w, grad_dtype=x.dtype)
    assert torch.equal(g["dx"][s], gs["dx"]) and torch.equal(g["dz"][s], gs["dz"])
    del g
    y, h, r, _ = gdr.residual_norm_fwd(x, x, w, gate=x)
    ys, hs, rs, _ = gdr.residual_norm_fwd(x[s], x[s], w, gate=x[s])
    assert torch.equal(y[s], ys) and torch.equal(h[s], hs) and torch.equal(r[s], rs)
    del y
    g = gdr.residual_norm_bwd(x, h, x, r, w, gate=x, grad_dtype=x.dtype)
    gs = gdr.residual_norm_bwd(x[s], hs, x[s], rs, w, gate=x[s], grad_dtype=x.dtype)
    assert all(torch.equal(g[k][s], gs[k]) for k in ("dx", "dresidual", "dgate"))


def test_empty_calls():
    z = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, r = gdr.gated_norm_fwd(z, z, w)
    g = gdr.gated_norm_bwd(z, z, z, r, w)
    assert y.shape == (0, 64) and not g["dweight"].any()
    y, h, r, xr = gdr.residual_norm_fwd(z, z, w, x_weight=w, gate=w)
    g = gdr.residual_norm_bwd(z, h, z, r, w, x_weight=w, x_rstd=xr, gate=w)
    assert y.shape == h.shape == (0, 64) and not g["dweight"].any() and not g["dx_weight"].any() and not g["dgate"].any()


@pytest.mark.parametrize("dtype,R,C", [("bf16", 5, 700), ("f32", 7, 900), ("bf16", 1100, 4500), ("f32", 1030, 6000), ("bf16", 301, 8192),
                                       ("bf16", 259, 12000), ("f32", 263, 9000), ("bf16", 2049, 2050), ("f32", 515, 2100)])
def test_rows_that_go_round_the_grid(dtype, R, C):
    """More rows than workgroups take at a time: rows alone give the same bits, and the parameters' gradients are sums over
    all rows."""
    c = residual_case(R, C, dtype, dtype, "f32", True, "token")
    x, res, w, xw, gate = (dev(c[k]) for k in ("x", "res", "w", "xw", "g"))
    kw = dict(x_weight=xw, scale=0.6)
    y, h, r, xr = gdr.residual_norm_fwd(x, res, w, gate=gate, **kw)
    n, nr = gdr.gated_norm_fwd(x, res, w)
    g = gdr.residual_norm_bwd(x, h, y, r, w, d_h=h, x_rstd=xr, gate=gate, **kw)
    gg = gdr.gated_norm_bwd(x, res, y, nr, w)
    for s in (slice(0, 1), slice(R // 2, R // 2 + 2), slice(R - 1, R)):
        ys, hs, rs, xs = gdr.residual_norm_fwd(x[s], res[s], w, gate=gate[s], **kw)
        assert torch.equal(ys, y[s]) and torch.equal(hs, h[s]) and torch.equal(rs, r[s]) and torch.equal(xs, xr[s])
        assert torch.equal(gdr.gated_norm_fwd(x[s], res[s], w)[0], n[s])
        gs = gdr.residual_norm_bwd(x[s], hs, ys, rs, w, d_h=hs, x_rstd=xs, gate=gate[s], **kw)
        assert all(torch.equal(gs[k], g[k][s]) for k in ("dx", "dresidual", "dgate"))
        gs = gdr.gated_norm_bwd(x[s], res[s], ys, nr[s], w)
        assert torch.equal(gs["dx"], gg["dx"][s]) and torch.equal(gs["dz"], gg["dz"][s])
    hat = f64(h) * f64(r)[:, None]
    close("dweight", g["dweight"], (f64(y) * hat).sum(0), np.abs(f64(y) * hat).sum(0), R + 30)
    xh, dh = f64(x) * f64(xr)[:, None], f64(g["dresidual"])
    m = float(np.float32(0.6)) * f64(gate) * dh
    # the gradient of h is itself rounded once to fp32 where it was written
    close("dx_weight", g["dx_weight"], (m * xh).sum(0), np.abs(m * xh).sum(0), R + 40)
