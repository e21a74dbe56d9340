"""The layer operators in the forms that a layer chains them in: fp32 output gradients for bf16 inputs, single tokens with
fp32 outputs, more packed sequences than a wavefront has lanes, q, k and v out of one projection."""
import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
import test_gpu_mixer as m
from mixer_bounds import check, scan_bounds
from mixer_common import U, randn

pytestmark = pytest.mark.gpu


def fine(t, seed=17):
    """fp32 values near t's that bf16 does not hold."""
    return t.float() + torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)) / 512


def bf16_cases(cases):
    return sorted(k for k, v in cases.items() if v["dtype"] == "bf16")


@pytest.mark.parametrize("grad", ["io", "f32"])
@pytest.mark.parametrize("case", bf16_cases(m.CONV))
def test_conv_bwd_of_fp32_gradients(case, grad, monkeypatch):
    plain = m.conv_case

    def finer(**kw):
        c = plain(**kw)
        return dict(c, d_y=fine(c["d_y"]), dl=fine(c["dl"]))
    monkeypatch.setattr(m, "conv_case", finer)
    m.test_conv_bwd(case, grad)


@pytest.mark.parametrize("grad", ["io", "f32"])
@pytest.mark.parametrize("case", bf16_cases(m.SCAN))
def test_scan_bwd_of_fp32_gradients(case, grad, monkeypatch):
    plain = m.scan_case
    monkeypatch.setattr(m, "scan_case", lambda **kw: (lambda c: dict(c, d_y=fine(c["d_y"])))(plain(**kw)))
    m.test_scan_bwd(case, grad)


@pytest.mark.parametrize("dtype,R,C", [c for c in m.NORM if c[0] == "bf16"])
def test_layer_norm_of_fp32_gradients(dtype, R, C, monkeypatch):
    plain = m.norm_case

    def finer(*a, **kw):
        x, w, b, dy = plain(*a, **kw)
        return x, w, b, fine(dy)
    monkeypatch.setattr(m, "norm_case", finer)
    m.test_layer_norm(dtype, R, C)


def test_fp32_gradients_past_the_caches():
    """As many bytes as go past the caches: the bits of two smaller calls."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, dy, w, h0 = new(2, 7000, 4100).bfloat16(), new(2, 7000, 4100), new(4100, 4), new(2, 3, 4100)
    assert 2 * 7000 * 4100 * (2 + 4 + 2) > 256 << 20 > 7000 * 4100 * (2 + 4 + 2)
    kw = dict(initial_state=h0.bfloat16(), d_final_state=h0, grad_dtype=x.dtype)
    g = gdr.conv_bwd(x, w, dy, **kw)
    for i in range(2):
        kw = dict(initial_state=h0[i:i + 1].bfloat16(), d_final_state=h0[i:i + 1], grad_dtype=x.dtype)
        p = gdr.conv_bwd(x[i:i + 1], w, dy[i:i + 1], **kw)
        assert torch.equal(p["dx"][0], g["dx"][i]) and torch.equal(p["dh0"][0], g["dh0"][i])
    x, dy, w = x.view(-1, 4100), dy.view(-1, 4100), w[:, 0].contiguous()
    _, mean, rstd = gdr.layer_norm_fwd(x, w)
    dx = gdr.layer_norm_bwd(x, dy, mean, rstd, w, grad_dtype=x.dtype)["dx"]
    for s in (slice(0, 6000), slice(6000, 14000)):
        assert torch.equal(dx[s], gdr.layer_norm_bwd(x[s], dy[s], mean[s], rstd[s], w, grad_dtype=x.dtype)["dx"])


@pytest.mark.parametrize("case", ["batch_groups", "strided", "state_7_odd", "state_50"])
def test_scan_step_fp32_outputs(case):
    c = m.scan_case(**dict(m.SCAN[case], lens=[1] * 5, batch=True))
    a, k = m.scan_args(c)
    one = lambda t: None if t is None else t[:, 0]
    out, states = [], []
    for dtype in (torch.float32, None):
        state = m.dev(c["h0"]).clone()
        out.append(gdr.scan_step(one(a[0]), one(a[1]), a[2], one(a[3]), one(a[4]), state, k["D"], one(k["z"]), k["dt_bias"],
                                 k["dt_softplus"], out_dtype=dtype))
        states.append(state)
    assert out[0].dtype == torch.float32 and torch.equal(out[0].bfloat16(), out[1]) and torch.equal(*states)
    ref, err = scan_bounds(c["ref"], c["pre"], c["soft"], c["zf"])
    check("y", out[0], ref["y"], err["y"], 3e-4)
    check("state", states[0], ref["last"], err["last"], 3e-4)


def many(N, seed):
    """N short ragged sequences, empty ones at the front, in the middle and at the end."""
    lens = np.random.default_rng(seed).integers(0, 4, N)
    lens[[0, 1, N // 2, N // 2 + 1, N - 2, N - 1]] = 0
    lens[N // 3] = 70
    return [int(v) for v in lens]


MANY_CONV = {
    "two_taps": dict(dtype="bf16", lens=[100, 0, 3], D=520, W=2),
    "64_of_them": dict(dtype="bf16", lens=many(64, 0), D=40, W=4),
    "65_of_them": dict(dtype="bf16", lens=many(65, 1), D=40, W=4),
    "200_of_them": dict(dtype="f32", lens=many(200, 2), D=13, W=3),
    "5000_of_them": dict(dtype="bf16", lens=many(5000, 3), D=24, W=4),
}
MANY_SCAN = {
    "64_of_them": dict(dtype="bf16", lens=many(64, 0), D=40, S=16),
    "65_of_them": dict(dtype="bf16", lens=many(65, 1), D=40, S=16),
    "200_of_them": dict(dtype="f32", lens=many(200, 2), D=18, S=24, G=2),
    "5000_of_them": dict(dtype="bf16", lens=many(5000, 3), D=16, S=8),
}


@pytest.mark.parametrize("case", sorted(MANY_CONV))
def test_conv_of_many_sequences(case, monkeypatch):
    monkeypatch.setitem(m.CONV, case, MANY_CONV[case])
    m.test_conv_fwd(case)
    m.test_conv_bwd(case, "f32")


@pytest.mark.parametrize("case", sorted(MANY_SCAN))
def test_scan_of_many_sequences(case):
    c = m.scan_case(**MANY_SCAN[case])
    n, D = len(c["pre"]), c["ref"]["A"].shape[0]
    ref, err = scan_bounds(c["ref"], c["pre"], c["soft"], c["zf"], m.f64(c["d_y"]).reshape(n, D), m.f64(c["dl"]))
    y, last = m.run_scan(c, out_dtype=torch.float32)
    got = dict(m.run_scan(c, back=True), y=y, last=last)
    for k in ref:
        check("%s %s" % (case, k), got[k], ref[k], err[k], {"dA": 2e-2, "dD": 2e-2, "ddt_bias": 5e-2}.get(k, 3e-4))


def test_the_readme_chain():
    """Norm, scan and convolution backward as the README chains them: scan_bwd's fp32 dx goes into conv_bwd of bf16 inputs."""
    gen = torch.Generator().manual_seed(2)
    B, T, D, S = 2, 150, 48, 16
    x, dt, z, d_o = (randn(gen, B, T, D, dtype=torch.bfloat16).cuda() for _ in range(4))
    Bm, Cm = (randn(gen, B, T, 1, S, dtype=torch.bfloat16).cuda() for _ in range(2))
    w, b, A = randn(gen, D, 4, std=0.5).cuda(), randn(gen, D).cuda(), -torch.exp(randn(gen, D, S)).cuda()
    kw = dict(z=z, dt_softplus=True)
    u, _ = gdr.conv_fwd(x, w, b)
    y, _ = gdr.scan_fwd(u, dt, A, Bm, Cm, **kw)
    _, mean, rstd = gdr.layer_norm_fwd(y)
    g = gdr.layer_norm_bwd(y, d_o, mean, rstd)
    gs = gdr.scan_bwd(u, dt, A, Bm, Cm, g["dx"], **kw)
    gc = gdr.conv_bwd(x, w, gs["dx"], b)
    assert g["dx"].dtype == gs["dx"].dtype == gc["dx"].dtype == torch.float32
    cu = np.arange(B + 1) * T
    n = B * T
    xf, wf, bf = m.f64(x).reshape(n, D), m.f64(w), m.f64(b)
    h0, dy = np.zeros((B, 3, D)), m.f64(gs["dx"]).reshape(n, D)
    p, _, _ = m.om.conv(xf, wf, bf, cu, h0, True)
    Mp, _, _ = m.om.conv(np.abs(xf), np.abs(wf), np.abs(bf), cu, h0, False)
    ref = m.om.conv_backward(xf, wf, dy * m.om.silu_grad(p), cu, h0, h0)
    M = m.om.conv_backward(np.abs(xf), np.abs(wf), np.abs(dy) * (2.0 + Mp), cu, h0, h0)
    for name, r, a, terms in zip(("dx", "dweight", "dbias"), ref, M, (5, n, n)):
        m.close(name, gc[name], r, a, 8 + 2 * np.abs(p).max() + 12 + terms)


def test_q_k_v_out_of_one_projection():
    """Three calls on slices of the projection give dense q, k and v, the bits of one call that is cut afterwards."""
    gen = torch.Generator().manual_seed(5)
    H, d = 2, 64
    cu = torch.tensor([0, 70, 70, 160], dtype=torch.int32)
    kw = dict(cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu)
    wide = randn(gen, 1, 160, 4 * H * d + 8, dtype=torch.bfloat16).cuda()
    x, w = wide[..., :4 * H * d], randn(gen, 4 * H * d, 4, std=0.5).cuda()
    ends = (0, H * d, 2 * H * d, 4 * H * d)
    whole, last = gdr.conv_fwd(x, w, **kw)
    parts = [gdr.conv_fwd(x[..., i:j], w[i:j], **kw) for i, j in zip(ends, ends[1:])]
    for (y, st), i, j in zip(parts, ends, ends[1:]):
        assert y.is_contiguous() and torch.equal(y, whole[..., i:j]) and torch.equal(st, last[..., i:j])
    beta = torch.sigmoid(randn(gen, 1, 160, 2 * H)).bfloat16().cuda()
    g = -torch.rand(1, 160, 2 * H, generator=gen).cuda()
    heads = lambda t: t.view(1, 160, -1, d)
    unit = lambda t: torch.nn.functional.normalize(heads(t).float(), dim=-1).to(t.dtype)
    q, k, v = (y for y, _ in parts)
    o, S = gdr.chunk_fwd(heads(q), unit(k), heads(v), beta, g=g, **kw)
    q, k, v = (whole[..., i:j].contiguous() for i, j in zip(ends, ends[1:]))
    o2, S2 = gdr.chunk_fwd(heads(q), unit(k), heads(v), beta, g=g, **kw)
    assert torch.isfinite(o).all() and torch.equal(o, o2) and torch.equal(S, S2)
