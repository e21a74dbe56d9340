"""Error bounds of the selective state space scan that follow it token by token: an error made at one token decays with
the state that carries it, so that long sequences are bounded as tightly as short ones.

U = 2^-24, half a step of fp32. In units of U, with pre = dt + dt_bias and delta the step size:
  delta            eta = 3 |pre| + 14 with softplus (2 |pre| + 12 of the function, |pre| + 1 of the rounded sum), else 1
  exp(delta A)     |delta A| (3 + eta) + 2: A log2 e (constant and product), times delta, the instruction
  a joined piece   P = exp(A sum(delta)): the sum's additions (a piece's 16 tokens, a segment's tiles and wavefronts:
                   64 at most for segments of up to 640 tokens) enter as |delta A| 64 a token
  a state          one rounding a token, one more a joined piece, one where both meet: 3 of its absolute sum H
  silu(z), silu'   2 |z| + 10, and of each of its terms 2 |z| + 12
Sums of n products add n of the sum of their absolute values, sums over the tokens n of the sum of |each token's value|
(whose own error counts besides). Everything below that starts with e is such an error.
"""
import numpy as np
import torch

from mixer_common import U, f64
from oracle import mixer as om

ADDS = 64


def _heads(v, D):
    return np.repeat(v, D // v.shape[-2], axis=-2)


def scan_bounds(r, pre, soft, zf=None, dy=None, dl=None):
    """(references, bounds in units of U) by output name, for r = dict(x, delta, A, B, C, skip, cu, h0) in float64, the
    gate's argument zf (or None) and, for the gradients, dL/dy and dL/dfinal_state."""
    x, delta, A, B, C, skip, cu, h0 = (r[k] for k in ("x", "delta", "A", "B", "C", "skip", "cu", "h0"))
    n, D = x.shape
    G, S = B.shape[1:]
    N = len(cu) - 1
    eta = 3 * np.abs(pre) + 14 if soft else np.ones_like(pre)
    gate = np.ones((n, D)) if zf is None else om.silu(zf)
    eg_ = np.zeros((n, D)) if zf is None else 2 * np.abs(zf) + 10         # relative error of the gate
    hs, Hs, es = (np.zeros((n, D, S)) for _ in range(3))
    last, elast = h0.copy(), np.zeros_like(h0)

    def factors(t):
        m = np.abs(delta[t][:, None] * A)
        return np.exp(delta[t][:, None] * A), m * (3 + ADDS + eta[t][:, None]) + 2
    for q in range(N):
        h, H, e = h0[q], np.abs(h0[q]), np.zeros((D, S))
        for t in range(cu[q], cu[q + 1]):
            a, ea = factors(t)
            b = (delta[t] * x[t])[:, None] * _heads(B[t], D)
            h, e, H = a * h + b, a * (e + ea * H) + (eta[t][:, None] + 3) * np.abs(b), a * H + np.abs(b)
            e = e + 3 * H
            hs[t], Hs[t], es[t] = h, H, e
        last[q], elast[q] = h, e
    Ch, aC = np.stack([_heads(c, D) for c in C]) if n else np.zeros((0, D, S)), None
    aC = np.abs(Ch)
    v, Mv = (Ch * hs).sum(2) + skip * x, (aC * Hs).sum(2) + np.abs(skip * x)
    ev = (aC * es).sum(2) + (S + 6) * Mv
    ref = dict(y=v * gate, last=last)
    err = dict(y=(ev + (eg_ + 2) * Mv) * np.abs(gate), last=elast)
    if dy is None:
        return ref, err
    ds, eds = dy * gate, eg_ + 1                            # eds: relative
    keys = ("dx", "ddt", "dB", "dC")
    out, oe = ({k: np.zeros(s) for k, s in zip(keys, ((n, D), (n, D), B.shape, B.shape))} for _ in range(2))
    dA, edA, MdA = (np.zeros_like(A) for _ in range(3))
    dh0, edh0 = np.zeros_like(h0), np.zeros_like(h0)
    slope = 1 / (1 + np.exp(-pre)) if soft else np.ones_like(pre)
    eslope = 3 * np.abs(pre) + 14 if soft else np.zeros_like(pre)
    group = lambda w: w.reshape(G, D // G, S).sum(1)
    for q in range(N):
        Gr, Gm, eG = dl[q], np.abs(dl[q]), np.zeros((D, S))
        for t in reversed(range(cu[q], cu[q + 1])):
            a, ea = factors(t)
            first = t == cu[q]
            hp, Hp, ep = (h0[q], np.abs(h0[q]), 0.0) if first else (hs[t - 1], Hs[t - 1], es[t - 1])
            dsC = ds[t][:, None] * Ch[t]
            g, gm = Gr + dsC, Gm + np.abs(dsC)
            eg = eG + (eds[t][:, None] + 1) * np.abs(dsC) + 3 * gm
            ads, dlt = np.abs(ds[t]), np.abs(delta[t])
            out["dC"][t], M = group(ds[t][:, None] * hs[t]), group(ads[:, None] * Hs[t])
            oe["dC"][t] = group(ads[:, None] * (es[t] + (eds[t][:, None] + 1) * Hs[t])) + (D // G + 4) * M
            dxt = (delta[t] * x[t])[:, None]
            out["dB"][t], M = group(g * dxt), group(gm * np.abs(dxt))
            oe["dB"][t] = group(np.abs(dxt) * (eg + (eta[t][:, None] + 2) * gm)) + (D // G + 4) * M
            Bh = _heads(B[t], D)
            gB, gBm = (g * Bh).sum(1), (gm * np.abs(Bh)).sum(1)
            egB = (np.abs(Bh) * eg).sum(1) + (S + 2) * gBm
            out["dx"][t] = delta[t] * gB + skip * ds[t]
            oe["dx"][t] = dlt * (egB + (eta[t] + 3) * gBm) + (eds[t] + 3) * np.abs(skip * ds[t])
            p, pm = a * hp, a * Hp
            epp = a * ep + (ea + 1) * pm
            gp, gpm, egp = g * p, gm * pm, eg * pm + gm * epp + 2 * gm * pm
            gAm = (gpm * np.abs(A)).sum(1)
            egA = (np.abs(A) * egp).sum(1) + (S + 6) * gAm
            ddelta, mdd = x[t] * gB + (gp * A).sum(1), np.abs(x[t]) * gBm + gAm
            out["ddt"][t] = ddelta * slope[t]
            oe["ddt"][t] = (np.abs(x[t]) * egB + egA + (4 + eslope[t]) * mdd) * slope[t]
            dA += gp * delta[t][:, None]
            edA += (egp + (eta[t][:, None] + 2) * gpm) * dlt[:, None]
            MdA += np.abs(gp) * dlt[:, None]
            Gr, Gm, eG = a * g, a * gm, a * (eg + (ea + 1) * gm)
        dh0[q], edh0[q] = Gr, eG
    ref.update(out, dA=dA, dD=(ds * x).sum(0), ddt_bias=out["ddt"].sum(0), dh0=dh0)
    err.update(oe, dA=edA + n * MdA, dD=((eds + n) * np.abs(ds * x)).sum(0),
               ddt_bias=oe["ddt"].sum(0) + n * np.abs(out["ddt"]).sum(0), dh0=edh0)
    if zf is not None:
        s = 1 / (1 + np.exp(-zf))
        terms = s * (1 + np.abs(zf) * (1 - s))
        ref["dz"] = dy * v * om.silu_grad(zf)
        err["dz"] = np.abs(dy) * terms * (ev + (2 * np.abs(zf) + 14) * Mv)
    return ref, err


def excess(got, ref, err, half=0.0):
    """The largest |got - ref| / bound; half: half a step of the stored type relative to the value."""
    bound = 1.02 * U * err * (1 + half) + half * np.abs(ref) + 1e-37
    return float((np.abs(got - ref) / bound).max()) if ref.size else 0.0


def share(ref, err):
    """The bound's median relative to the outputs' root mean square."""
    return float(np.median(U * err) / np.sqrt(np.mean(ref ** 2))) if ref.size else 0.0


def check(name, got, ref, err, most):
    """got lies within the bound, and the bound says something: its median is at most `most` of the outputs' size."""
    half = torch.finfo(got.dtype).eps / 2
    worst, tight = excess(f64(got).reshape(ref.shape), ref, err, half), share(ref, err)
    print("%s: worst error / bound %.3f, bound / size %.1e" % (name, worst, tight), flush=True)
    assert np.isfinite(f64(got)).all(), name
    assert worst <= 1.0 and tight <= most, (name, worst, tight)
