"""Pins of oracle/mixer.py: closed forms, independent library forms in float64
and central differences of every gradient."""
import numpy as np
import pytest
import torch

from oracle import mixer as om

CU = np.array([0, 1, 1, 4, 9])              # lengths 1, 0, 3, 5


def rand(rng, *shape):
    return rng.standard_normal(shape)


def differences(f, arrays, grads, rng, eps=1e-6, tol=1e-6):
    """<grad, direction> against the central difference of f along a random direction of each array."""
    for name, arr in arrays.items():
        d = rng.standard_normal(arr.shape)
        keep = arr.copy()
        arr[...] = keep + eps * d
        hi = f()
        arr[...] = keep - eps * d
        lo = f()
        arr[...] = keep
        want, got = (hi - lo) / (2 * eps), float((grads[name] * d).sum())
        assert abs(want - got) <= tol * max(1.0, abs(want)), (name, want, got)


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_matches_torch_and_differences(W):
    rng = np.random.default_rng(W)
    n, D, N = int(CU[-1]), 5, len(CU) - 1
    x, w, b, h0 = rand(rng, n, D), rand(rng, D, W), rand(rng, D), rand(rng, N, W - 1, D)
    p, y, last = om.conv(x, w, b, CU, h0, True)
    for q in range(N):
        s, e = CU[q], CU[q + 1]
        u = torch.tensor(np.concatenate([h0[q], x[s:e]]).T[None])
        if e > s:
            ref = torch.nn.functional.conv1d(u, torch.tensor(w)[:, None], torch.tensor(b), groups=D)[0].T.numpy()
            assert np.allclose(p[s:e], ref, atol=1e-12)
            assert np.allclose(y[s:e], torch.nn.functional.silu(torch.tensor(ref)).numpy(), atol=1e-12)
        assert np.array_equal(last[q], u[0].T.numpy()[-(W - 1):])
    cy, cl = rand(rng, n, D), rand(rng, N, W - 1, D)

    def loss():
        _, y, last = om.conv(x, w, b, CU, h0, True)
        return float((y * cy).sum() + (last * cl).sum())
    dx, dw, db, dh0 = om.conv_backward(x, w, cy * om.silu_grad(p), CU, h0, cl)
    differences(loss, dict(x=x, w=w, b=b, h0=h0), dict(x=dx, w=dw, b=db, h0=dh0), rng)


def test_scan_closed_form_and_differences():
    rng = np.random.default_rng(7)
    n, D, G, S, N = int(CU[-1]), 6, 2, 3, len(CU) - 1
    x, delta = rand(rng, n, D), np.abs(rand(rng, n, D)) * 0.5
    A, B, C = -np.abs(rand(rng, D, S)), rand(rng, n, G, S), rand(rng, n, G, S)
    skip, h0 = rand(rng, D), rand(rng, N, D, S)
    v, hs, last = om.scan(x, delta, A, B, C, skip, CU, h0)
    q, d, s = 3, 4, 1                           # the sum over earlier tokens written out
    for t in range(CU[q], CU[q + 1]):
        want = np.exp(A[d, s] * delta[CU[q]:t + 1, d].sum()) * h0[q, d, s]
        for r in range(CU[q], t + 1):
            want += np.exp(A[d, s] * delta[r + 1:t + 1, d].sum()) * delta[r, d] * B[r, d // 3, s] * x[r, d]
        assert abs(hs[t, d, s] - want) < 1e-12
    assert np.array_equal(last[1], h0[1])       # the empty sequence
    cv, cl = rand(rng, n, D), rand(rng, N, D, S)

    def loss():
        v, _, last = om.scan(x, delta, A, B, C, skip, CU, h0)
        return float((v * cv).sum() + (last * cl).sum())
    names = ("x", "delta", "A", "B", "C", "skip", "h0")
    grads = dict(zip(names, om.scan_backward(x, delta, A, B, C, skip, CU, h0, cv, cl)))
    differences(loss, dict(x=x, delta=delta, A=A, B=B, C=C, skip=skip, h0=h0), grads, rng)


def test_layer_norm_matches_torch_and_differences():
    rng = np.random.default_rng(9)
    x, w, b = rand(rng, 4, 7), rand(rng, 7), rand(rng, 7)
    y, mean, rstd = om.layer_norm(x, w, b, 1e-5)
    ref = torch.nn.functional.layer_norm(torch.tensor(x), (7,), torch.tensor(w), torch.tensor(b), 1e-5).numpy()
    assert np.allclose(y, ref, atol=1e-12)
    cy = rand(rng, 4, 7)
    dx, dw, db = om.layer_norm_backward(x, cy, mean, rstd, w)
    differences(lambda: float((om.layer_norm(x, w, b, 1e-5)[0] * cy).sum()), dict(x=x, w=w, b=b),
                dict(x=dx, w=dw, b=db), rng)


def test_activations():
    v = np.linspace(-30, 30, 61)
    t = torch.tensor(v, requires_grad=True)
    torch.nn.functional.silu(t).sum().backward()
    assert np.allclose(om.silu_grad(v), t.grad.numpy(), atol=1e-14)
    assert np.allclose(om.softplus(v), torch.nn.functional.softplus(torch.tensor(v), threshold=1e9).numpy(), rtol=1e-14)
