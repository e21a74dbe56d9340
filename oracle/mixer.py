"""The layer operators next to the gated delta rule, in float64 from their
definitions: the short causal convolution, the selective state space scan (token
by token) and layer norm, each with its gradients written out.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Tokens are flattened; ``cu`` are the sequence offsets. The scan's functions take
the step sizes delta themselves (softplus and bias are the caller's), so that
the same code run on absolute values bounds every sum of products: a GPU result
whose factors carry a relative error e each is off by at most (number of
factors) e times that bound.
"""
from __future__ import annotations

import numpy as np


def silu(p):
    return p / (1.0 + np.exp(-p))


def silu_grad(p):
    s = 1.0 / (1.0 + np.exp(-p))
    return s * (1.0 + p * (1.0 - s))


def softplus(v):
    return np.logaddexp(0.0, v)


def conv_taps(x, cu, h0, W):
    """win[t, w] = u_{t-(W-1)+w}, and every sequence's last W - 1 rows of u."""
    n, D = x.shape
    win, last = np.zeros((n, W, D)), np.zeros((len(cu) - 1, W - 1, D))
    for q in range(len(cu) - 1):
        s, e = cu[q], cu[q + 1]
        u = np.concatenate([h0[q], x[s:e]])
        for w in range(W):
            win[s:e, w] = u[w:w + e - s]
        last[q] = u[e - s:]
    return win, last


def conv(x, weight, bias, cu, h0, act):
    """p (pre-activation), y, final state; weight [D, W]."""
    win, last = conv_taps(x, cu, h0, weight.shape[1])
    p = np.einsum("twd,dw->td", win, weight) + bias
    return p, (silu(p) if act else p), last


def conv_backward(x, weight, dp, cu, h0, d_last):
    """dx, dweight, dbias, dh0 for the pre-activation's gradient dp."""
    D, W = weight.shape
    win, _ = conv_taps(x, cu, h0, W)
    dx, dh0 = np.zeros_like(x), np.zeros_like(h0)
    for q in range(len(cu) - 1):
        s, e = cu[q], cu[q + 1]
        du = np.zeros((W - 1 + e - s, D))
        du[e - s:] += d_last[q]
        for w in range(W):
            du[w:w + e - s] += dp[s:e] * weight[:, w]
        dh0[q], dx[s:e] = du[:W - 1], du[W - 1:]
    return dx, np.einsum("td,twd->dw", dp, win), dp.sum(0), dh0


def _heads(v, D):
    return np.repeat(v, D // v.shape[-2], axis=-2)          # [G, S] -> [D, S]


def scan(x, delta, A, B, C, skip, cu, h0):
    """v (before the gate) [T, D], states after every token [T, D, S], final states."""
    n, D = x.shape
    v, hs, last = np.zeros((n, D)), np.zeros((n, D, A.shape[1])), h0.copy()
    for q in range(len(cu) - 1):
        h = h0[q].copy()
        for t in range(cu[q], cu[q + 1]):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * _heads(B[t], D)
            hs[t] = h
            v[t] = (_heads(C[t], D) * h).sum(1) + skip * x[t]
        last[q] = h
    return v, hs, last


def scan_backward(x, delta, A, B, C, skip, cu, h0, ds, d_last, factor_A=None):
    """Gradients for ds = dL/dv: dx, ddelta, dA, dB, dC, dskip, dh0.
    factor_A replaces A where it stands as a factor (absolute values)."""
    n, D = x.shape
    G, S = B.shape[1:]
    fA = A if factor_A is None else factor_A
    _, hs, _ = scan(x, delta, A, B, C, skip, cu, h0)
    dx, dd, dB, dC = np.zeros_like(x), np.zeros_like(x), np.zeros_like(B), np.zeros_like(C)
    dA, dh0 = np.zeros_like(A), np.zeros_like(h0)
    for q in range(len(cu) - 1):
        g = d_last[q].copy()
        for t in reversed(range(cu[q], cu[q + 1])):
            prev = hs[t - 1] if t > cu[q] else h0[q]
            a = np.exp(delta[t][:, None] * A)
            g = g + ds[t][:, None] * _heads(C[t], D)
            dC[t] = (ds[t][:, None] * hs[t]).reshape(G, D // G, S).sum(1)
            dB[t] = ((delta[t] * x[t])[:, None] * g).reshape(G, D // G, S).sum(1)
            gB = (g * _heads(B[t], D)).sum(1)
            gp = g * a * prev
            dx[t] = delta[t] * gB + skip * ds[t]
            dd[t] = x[t] * gB + (gp * fA).sum(1)
            dA += gp * delta[t][:, None]
            g = a * g
        dh0[q] = g
    return dx, dd, dA, dB, dC, (ds * x).sum(0), dh0


def layer_norm(x, weight, bias, eps):
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(-1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * weight + bias, mean, rstd


def layer_norm_backward(x, dy, mean, rstd, weight):
    hat = (x - mean[:, None]) * rstd[:, None]
    c = dy * weight
    dx = rstd[:, None] * (c - c.mean(-1, keepdims=True) - hat * (c * hat).mean(-1, keepdims=True))
    return dx, (dy * hat).sum(0), dy.sum(0)
