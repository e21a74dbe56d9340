"""oracle/attn.py and oracle/block_norm.py against other forms of the definitions and against differences."""
import numpy as np
import pytest

from oracle import attn as oa
from oracle import block_norm as ob


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (4, 0), (3, 1), (5, 9), (50, 3)])
def test_attend_is_softmax_over_what_is_seen(window, sinks):
    rng = np.random.default_rng(window * 10 + sinks)
    n, dk, dv = 14, 5, 3
    q, k, v = rng.standard_normal((n, dk)), rng.standard_normal((n, dk)), rng.standard_normal((n, dv))
    o, lse, _ = oa.attend(q, k, v, np.arange(n), np.arange(n), window, sinks, 0.7)
    for p in range(n):
        js = [j for j in range(p + 1) if j > p - window or j < sinks]
        w = np.array([np.exp(0.7 * q[p] @ k[j]) for j in js])
        assert np.allclose(o[p], sum(x * v[j] for x, j in zip(w, js)) / w.sum())
        assert np.isclose(lse[p], np.log(w.sum()))


@pytest.mark.parametrize("window,sinks", [(1, 0), (4, 0), (3, 1), (5, 9), (2, 3)])
def test_caches_hold_what_later_tokens_see(window, sinks):
    """Token by token from the cache gives what the whole sequence gives, from any length on."""
    rng = np.random.default_rng(window + 100 * sinks)
    n, d = 17, 4
    q, k, v = (rng.standard_normal((n, d)) for _ in range(3))
    whole, _, _ = oa.attend(q, k, v, np.arange(n), np.arange(n), window, sinks, 0.5)
    kc, vc = np.full((sinks + window, d), np.nan), np.full((sinks + window, d), np.nan)
    for t in range(n):
        old = oa.cached_positions(t, window, sinks)
        at = [oa.slot(p, window, sinks) for p in old]
        o, _, _ = oa.attend(q[t:t + 1], np.concatenate([kc[at], k[t:t + 1]]), np.concatenate([vc[at], v[t:t + 1]]),
                            np.array([t]), np.array(old + [t]), window, sinks, 0.5)
        assert np.allclose(o[0], whole[t])
        kc, vc = oa.keep(kc, k[t:t + 1], t, window, sinks), oa.keep(vc, v[t:t + 1], t, window, sinks)


def differences(f, x, g, step=1e-6):
    """Gradient of sum(f() * g) with respect to x, an array that f reads."""
    out = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i, old = it.multi_index, x[it.multi_index]
        x[i] = old + step
        hi = sum((a * b).sum() for a, b in zip(f(), g))
        x[i] = old - step
        lo = sum((a * b).sum() for a, b in zip(f(), g))
        x[i] = old
        out[i] = (hi - lo) / (2 * step)
    return out


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (20, 0)])
def test_attention_gradients(window, sinks):
    rng = np.random.default_rng(window)
    n = 9
    q, k, v = rng.standard_normal((n, 4)), rng.standard_normal((n, 4)), rng.standard_normal((n, 3))
    pos, g = np.arange(n), rng.standard_normal((n, 3))
    f = lambda: [oa.attend(q, k, v, pos, pos, window, sinks, 0.6)[0]]
    o, lse, _ = oa.attend(q, k, v, pos, pos, window, sinks, 0.6)
    for x, d in zip((q, k, v), oa.attend_backward(q, k, v, o, lse, g, pos, pos, window, sinks, 0.6)):
        assert np.allclose(d, differences(f, x, [g]), atol=1e-7)


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gated_norm_gradients(act):
    rng = np.random.default_rng(1)
    x, z, w, g = (rng.standard_normal(s) for s in ((4, 7), (4, 7), (7,), (4, 7)))
    f = lambda: [ob.gated_norm(x, z, w, act, 0.1)[0]]
    r = ob.rstd(x, 0.1)
    assert np.allclose(f()[0][2, 3], x[2, 3] / np.sqrt((x[2] ** 2).mean() + 0.1) * w[3] * ob.gate(z, act)[2, 3])
    for a, d in zip((x, z, w), ob.gated_norm_backward(x, z, g, r, w, act)):
        assert np.allclose(d, differences(f, a, [g]), atol=1e-7)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("kind", ["none", "channel", "token"])
def test_residual_norm_gradients(post, kind):
    rng = np.random.default_rng(2)
    R, C = 3, 6
    x, res, w, gy, gh = (rng.standard_normal(s) for s in ((R, C), (R, C), (C,), (R, C), (R, C)))
    xw = rng.standard_normal(C) if post else None
    g = {"none": np.ones(()), "channel": rng.standard_normal(C), "token": rng.standard_normal((R, C))}[kind]
    f = lambda: ob.residual_norm(x, res, w, xw, g, 0.4, 0.05)[:2]
    _, h, r, xr = ob.residual_norm(x, res, w, xw, g, 0.4, 0.05)
    d = ob.residual_norm_backward(x, h, gy, gh, r, xr, w, xw, g, 0.4)
    assert np.allclose(d["dx"], differences(f, x, [gy, gh]), atol=1e-7)
    assert np.allclose(d["dresidual"], differences(f, res, [gy, gh]), atol=1e-7)
    assert np.allclose(d["dweight"], differences(f, w, [gy, gh]), atol=1e-7)
    if post:
        assert np.allclose(d["dx_weight"], differences(f, xw, [gy, gh]), atol=1e-7)
    if kind != "none":
        dg = d["dgate"] if kind == "token" else d["dgate"].sum(0)
        assert np.allclose(dg, differences(f, g, [gy, gh]), atol=1e-7)
