"""The window attention, the gated norm and the residual sum together, as a model uses them: a block of window attention
and one of the gated delta rule behind each other, prompts, single tokens, captured, and with their gradients."""
import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from attn_common import backward_reference, forward_reference, within
from mixer_common import U, close, f64, randn
from oracle import block_norm as ob

pytestmark = pytest.mark.gpu

D, NQ, NK, HD, W, S = 256, 4, 2, 64, 24, 3
EPS, SCALE = 1e-5, 0.75


class Weights:
    def __init__(self, dtype, seed=0):
        gen = torch.Generator().manual_seed(seed)
        new = lambda *s, mean=0.0, std=1.0, dtype=dtype: randn(gen, *s, dtype=dtype, mean=mean, std=std).cuda()
        self.qkv = new(D, (NQ + 2 * NK) * HD, std=D ** -0.5)
        self.z = new(D, NQ * HD, std=D ** -0.5)
        self.out = new(NQ * HD, D, std=(NQ * HD) ** -0.5)
        self.delta = new(D, 2 * NQ * HD + NK * HD + 2 * NQ, std=D ** -0.5)
        self.back = new(NQ * HD, D, std=(NQ * HD) ** -0.5)
        norm = lambda n: new(n, mean=1.0, std=0.1, dtype=torch.float32)
        self.norm, self.behind, self.next, self.heads, self.last = norm(D), norm(D), norm(D), norm(HD), norm(D)


def split(p):
    """q, k, v of a projection's columns, without a copy"""
    a, b = NQ * HD, (NQ + NK) * HD
    return p[..., :a].unflatten(-1, (NQ, HD)), p[..., a:b].unflatten(-1, (NK, HD)), p[..., b:].unflatten(-1, (NK, HD))


def attention_block(w, x, res, gate, attend):
    """x, res [..., D] -> the next block's input, the residual stream, and what the gradients need"""
    y, h, r, xr = gdr.residual_norm_fwd(x, res, w.norm, x_weight=w.behind, gate=gate, scale=SCALE, eps=EPS)
    p = y @ w.qkv
    o, lse = attend(*split(p))
    z = (y @ w.z).unflatten(-1, (NQ, HD))
    n, nr = gdr.gated_norm_fwd(o, z, w.heads, eps=EPS)
    u = n.flatten(-2) @ w.out
    y2, h2, r2, _ = gdr.residual_norm_fwd(u, h, w.next, eps=EPS)
    return y2, h2, dict(y=y, h=h, r=r, xr=xr, p=p, o=o, lse=lse, z=z, n=n, nr=nr, u=u, r2=r2)


def delta_block(w, y, h, state=None, cu=None, cu_cpu=None):
    """The gated delta rule over the same heads, its gate, and the last norm"""
    p = y @ w.delta
    a, b, c = NK * HD, (NK + NQ) * HD, (NK + 2 * NQ) * HD
    k = torch.nn.functional.normalize(p[..., :a].unflatten(-1, (NK, HD)).float(), dim=-1).to(y.dtype)
    v, z = p[..., a:b].unflatten(-1, (NQ, HD)).contiguous(), p[..., b:c].unflatten(-1, (NQ, HD)).contiguous()
    beta, g = torch.sigmoid(p[..., c:c + NQ].float()), -torch.nn.functional.softplus(p[..., c + NQ:].float())
    o, state = gdr.chunk_fwd(k, k, v, beta, g=g, initial_state=state, cu_seqlens=cu, cu_seqlens_cpu=cu_cpu)
    n, _ = gdr.gated_norm_fwd(o, z, w.heads, activation="sigmoid", eps=EPS)
    out, h, _, _ = gdr.residual_norm_fwd(n.flatten(-2) @ w.back, h, w.last, eps=EPS)
    return out, h, state


def inputs(dtype, *lead, seed=1):
    gen = torch.Generator().manual_seed(seed)
    new = lambda std: randn(gen, *lead, D, dtype=dtype, std=std).cuda()
    return new(1.0), new(2.0), new(0.5)                # a block's output, the stream, a gate per token


def case_of(t, lens, dtype, cu):
    """What tests/attn_common.py takes, from the tensors of the run"""
    q, k, v = (x.cpu() for x in split(t["p"]))
    return dict(q=q, k=k, v=v, cu=cu, lens=list(lens), window=W, sinks=S, scale=HD ** -0.5, past=[0] * len(lens), cache=None,
                dims=(NQ, NK, HD, HD))


def check_norms(t, w, x, res, gate):
    """Each norm of the run on the tensors that it was given"""
    X, R, G = (f64(a).reshape(-1, D) for a in (x, res, gate))
    s = float(np.float32(SCALE))
    ry, rh, rr, rx = ob.residual_norm(X, R, f64(w.norm), f64(w.behind), G, s, EPS)
    Mh = np.abs(R) + s * np.abs(G * X * rx[:, None] * f64(w.behind))
    Ms = (Mh * np.abs(rh)).mean(-1) * rr ** 2
    close("h", t["h"], rh, Mh, D + 40)
    close("y", t["y"], ry, (Mh + np.abs(rh) * (1 + 2 * Ms[:, None])) * rr[:, None] * np.abs(f64(w.norm)), D + 60)
    O, Z = f64(t["o"]).reshape(-1, HD), f64(t["z"]).reshape(-1, HD)
    rn, _ = ob.gated_norm(O, Z, f64(w.heads), "silu", EPS)
    close("n", t["n"], rn, np.abs(rn), HD + 30 + 2 * np.abs(Z).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompts(dtype):
    """Packed prompts through both blocks; each of the new operators against its oracle on what the run gave it."""
    lens = [45, 0, 70, 1]
    cu = torch.tensor([0, 45, 45, 115, 116], dtype=torch.int32)
    w = Weights(dtype)
    x, res, gate = inputs(dtype, 1, 116)
    kw = dict(cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu)
    y, h, t = attention_block(w, x, res, gate, lambda q, k, v: gdr.window_attn_fwd(q, k, v, W, S, **kw))
    check_norms(t, w, x, res, gate)
    o, lse, eo, el, _ = forward_reference(case_of(t, lens, dtype, cu))
    within("o", t["o"], o, eo)
    within("lse", t["lse"], lse, el)
    out, h, _ = delta_block(w, y, h, cu=kw["cu_seqlens"], cu_cpu=cu)
    assert torch.isfinite(out.float()).all() and torch.isfinite(h.float()).all() and out.shape == x.shape


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_prompt_and_then_tokens(dtype):
    """A prompt, a piece of it and single tokens over a cache: each operator against its oracle for the whole sequences, on
    what the run gave it."""
    N, n = 2, 60
    w = Weights(dtype)
    x, res, gate = inputs(dtype, N, n)
    cache = tuple(torch.full((N, S + W, NK, HD), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    lens = torch.zeros(N, dtype=torch.int32, device="cuda")
    parts = []
    for a, b in ((0, 25), (25, 38)):
        part = [z[:, a:b].contiguous() for z in (x, res, gate)]
        parts.append(attention_block(w, *part, lambda q, k, v: gdr.window_attn_fwd(q, k, v, W, S, cache=cache, lens=lens))[2])
        lens += b - a
    for i in range(38, n):
        part = [z[:, i].contiguous() for z in (x, res, gate)]
        t = attention_block(w, *part, lambda q, k, v: (gdr.window_attn_step(q, k, v, cache, lens, W, S), None))[2]
        parts.append({k: None if v is None else v[:, None] for k, v in t.items()})
        lens += 1
    t = {k: torch.cat([a[k] for a in parts], 1) for k in ("y", "h", "p", "o", "z", "n")}
    check_norms(t, w, x, res, gate)
    o, _, eo, _, _ = forward_reference(case_of(t, [n] * N, dtype, None))
    within("o", t["o"], o, eo)
    k, v = split(t["p"])[1:]
    for pos in (0, 1, 2, 59, 58, 40, 36):
        at = pos if pos < S else S + (pos - S) % W
        assert torch.equal(cache[0][:, at], k[:, pos]) and torch.equal(cache[1][:, at], v[:, pos]), pos


def test_captured_decoding():
    """A captured step of the block, replayed between eager work, against eager steps bit for bit."""
    N = 3
    w = Weights(torch.bfloat16)
    gen = torch.Generator().manual_seed(5)
    cache = tuple(randn(gen, N, S + W, NK, HD, dtype=torch.bfloat16).cuda() for _ in range(2))
    copy = tuple(c.clone() for c in cache)
    lens = torch.tensor([0, 10, 500], dtype=torch.int32, device="cuda")
    lens2 = lens.clone()
    x, res, gate = inputs(torch.bfloat16, N)
    step = lambda cache, lens: attention_block(w, x, res, gate, lambda q, k, v: (gdr.window_attn_step(q, k, v, cache, lens, W, S), None))
    scratch = tuple(c.clone() for c in cache)
    step(scratch, lens)                                 # the library's own buffers before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, h, _ = step(cache, lens)
        lens.add_(1)
    for turn in range(5):
        for a, b in zip((x, res, gate), inputs(torch.bfloat16, N, seed=10 + turn)):
            a.copy_(b)
        g.replay()
        want, wh, _ = step(copy, lens2)
        lens2 += 1
        assert torch.equal(out, want) and torch.equal(h, wh) and torch.equal(lens, lens2), turn
        assert all(torch.equal(a, b) for a, b in zip(cache, copy)), turn
        torch.cuda.synchronize()


def block_gradients(w, t, h2, x, gate, dy2, dh2, cu):
    """The block's backward pass by the operators' own; products by hand"""
    g2 = gdr.residual_norm_bwd(t["u"], h2, dy2, t["r2"], w.next, d_h=dh2)
    dn = (g2["dx"].to(w.out.dtype) @ w.out.t()).unflatten(-1, (NQ, HD))
    gn = gdr.gated_norm_bwd(t["o"], t["z"], dn, t["nr"], w.heads)
    q, k, v = split(t["p"])
    ga = gdr.window_attn_bwd(q, k, v, t["o"], t["lse"], gn["dx"], W, S, **cu)
    dp = torch.cat([ga[a].flatten(-2) for a in ("dq", "dk", "dv")], -1)
    dy = dp.to(w.qkv.dtype) @ w.qkv.t() + gn["dz"].flatten(-2).to(w.z.dtype) @ w.z.t()
    g1 = gdr.residual_norm_bwd(x, t["h"], dy, t["r"], w.norm, d_h=g2["dresidual"], x_weight=w.behind, x_rstd=t["xr"], gate=gate,
                               scale=SCALE)
    return dict(x=g1["dx"], res=g1["dresidual"], gate=g1["dgate"], norm=g1["dweight"], behind=g1["dx_weight"], heads=gn["dweight"],
                next=g2["dweight"]), ga, gn


def test_gradients():
    """fp32: attention's gradients on what the run gave it within their bounds, and the gradient of a loss of the whole
    block along random directions against differences (the slope of 2 steps of 1e-2 / sqrt(elements): their third order
    and the loss's rounding are below 2e-3 of |gradient| |direction|)."""
    lens, cu = [70, 33], torch.tensor([0, 70, 103], dtype=torch.int32)
    kw = dict(cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu)
    w = Weights(torch.float32)
    x, res, gate = inputs(torch.float32, 1, 103)
    attend = lambda q, k, v: gdr.window_attn_fwd(q, k, v, W, S, **kw)
    y2, h2, t = attention_block(w, x, res, gate, attend)
    gen = torch.Generator().manual_seed(7)
    dy2, dh2 = randn(gen, 1, 103, D).cuda(), randn(gen, 1, 103, D).cuda()
    grads, ga, gn = block_gradients(w, t, h2, x, gate, dy2, dh2, kw)
    c = case_of(t, lens, torch.float32, cu)
    c["d_o"] = gn["dx"].cpu()
    ref = backward_reference(c, f64(t["o"]).reshape(-1, NQ, HD), f64(t["lse"]).reshape(-1, NQ))
    for a in ("dq", "dk", "dv"):
        within(a, ga[a], *ref[a])
    values = dict(x=x, res=res, gate=gate, norm=w.norm, behind=w.behind, heads=w.heads, next=w.next)
    loss = lambda: (lambda y, h, _: float((y.double() * dy2.double()).sum() + (h.double() * dh2.double()).sum()))(
        *attention_block(w, x, res, gate, attend))
    for name, value in values.items():
        g = grads[name].double()
        way = torch.randn(value.shape, generator=gen).cuda() / value.numel() ** 0.5 + (g / g.norm()).float()
        keep, step = value.clone(), 1e-2
        value.copy_(keep + step * way)
        up = loss()
        value.copy_(keep - step * way)
        down = loss()
        value.copy_(keep)
        slope, along = (up - down) / (2 * step), float((g * way.double()).sum())
        limit = 2e-3 * float(g.norm()) * float(way.norm())
        print("%s: slope %.6g, along the gradient %.6g, limit %.2g" % (name, slope, along, limit))
        assert abs(slope - along) <= limit, name
