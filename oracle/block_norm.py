"""The gated RMS norm and the residual sum with its norms in float64 from their
definitions, with their gradients written out.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import numpy as np


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def gate(z, act):
    return z * sigmoid(z) if act == "silu" else sigmoid(z)


def gate_slope(z, act):
    s = sigmoid(z)
    return s * (1.0 + z * (1.0 - s)) if act == "silu" else s * (1.0 - s)


def rstd(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1) + eps)


def rms_backward(c, hat, r):
    """Gradient with respect to x of sum(c * hat), hat = x r."""
    return r[:, None] * (c - hat * (c * hat).mean(-1, keepdims=True))


def gated_norm(x, z, w, act, eps):
    r = rstd(x, eps)
    return x * r[:, None] * w * gate(z, act), r


def gated_norm_backward(x, z, dy, r, w, act):
    """dx, dz, dweight"""
    hat = x * r[:, None]
    da = dy * gate(z, act)
    return rms_backward(da * w, hat, r), dy * hat * w * gate_slope(z, act), (da * hat).sum(0)


def residual_norm(x, res, w, xw, g, scale, eps):
    """y, h, rstd, x_rstd (None without xw); g: a number, [C] or [rows, C]."""
    xr = None if xw is None else rstd(x, eps)
    a = x if xw is None else x * xr[:, None] * xw
    h = res + scale * g * a
    r = rstd(h, eps)
    return h * r[:, None] * w, h, r, xr


def residual_norm_backward(x, h, dy, dh_in, r, xr, w, xw, g, scale):
    """dict dx, dresidual, dweight, dx_weight (with xw), dgate by token"""
    hat = h * r[:, None]
    dh = dh_in + rms_backward(dy * w, hat, r)
    out = dict(dresidual=dh, dweight=(dy * hat).sum(0))
    m = scale * g * dh
    if xw is None:
        out["dx"], a = m, x
    else:
        xhat = x * xr[:, None]
        out["dx"], a = rms_backward(m * xw, xhat, xr), xhat * xw
        out["dx_weight"] = (m * xhat).sum(0)
    out["dgate"] = scale * dh * a
    return out
