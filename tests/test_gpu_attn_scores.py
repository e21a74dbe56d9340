"""Window attention on the GPU where scores are large or infinite: what a token's scores may change, and values.

Values. q of some rows and all of k are whole numbers, those of q times 2^e, and scale is a power of two: the scores are
exact in fp32 in whatever order they are summed (64 or 128 products of at most 2 x 2), and apart from each other by
2^e scale >= 512 or equal. Weights then are 1 / ties to the highest keys and 0 < exp(-512) to all others, however large
the scores. With U = 2^-24 and half as in attn_common:
  o      the mean of the tied v: weights of one value w (rounded once) over their sum of up to 600 terms: half + 40 U
  lse    top + log(ties): scaling by c, its roundings, ln 2 and the sum: 8 U |lse| + 40 U
  P      in the gradients 1 / ties up to e = 40 U (and 8 U |lse| up to |lse| of 1024 ln 2), then as in attn_common: dS up to
         P ((e + half) |dP - delta| + ((dv + 4) U + half') M) (1 + half)
Rows between them, whose q is small, have the errors of attn_common.
"""
import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from attn_common import _weight_error, attn_case, half_of, sequences, within
from mixer_common import T, U, f64
from oracle import attn as oa
from test_gpu_attn import dev, run_bwd, run_fwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Nq", [2, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("factor", [300.0, 1e8, float("inf"), float("-inf")])
def test_a_key_changes_nothing_for_those_that_do_not_see_it(dtype, factor, Nq):
    """k of a token a few hundred times larger, far beyond 2^24, or infinite: all other tokens and the other key head's
    queries keep their bits, o and lse."""
    lens, window, sinks = [150, 380, 40], 50, 3
    c = attn_case(dtype, lens, Nq, 2, 64, 64, window, sinks)
    base, bl, _ = run_fwd(c)
    off, G = np.concatenate([[0], np.cumsum(lens)]), Nq // 2
    for n, j in ((1, 100), (1, 1), (1, 379), (0, 149), (2, 0), (2, 17)):
        d = dict(c, k=c["k"].clone())
        d["k"][0, off[n] + j, 0] *= factor
        o, lse, _ = run_fwd(d)
        p = np.arange(lens[n])
        hit = np.zeros(off[-1], bool)
        hit[off[n]:off[n + 1]] = (p >= j) & ((p - j < window) | (j < sinks))
        hit = torch.tensor(hit).cuda()
        assert torch.equal(o[0, ~hit], base[0, ~hit]) and torch.equal(lse[0, ~hit], bl[0, ~hit]), (n, j)
        assert torch.equal(o[0, :, G:], base[0, :, G:]) and torch.equal(lse[0, :, G:], bl[0, :, G:]), (n, j)
        assert not torch.equal(lse[0, hit][:, :G], bl[0, hit][:, :G]), (n, j)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("factor", [300.0, 1e8, float("inf")])
def test_a_query_changes_nothing_for_the_others(dtype, factor):
    """q of one head of one token larger or infinite: the token's other heads and all other tokens keep their bits, in a
    prompt of few rows, of many, and as single tokens."""
    for lens, Nq in (([60], 4), ([600], 64)):
        c = attn_case(dtype, lens, Nq, 1, 64, 64, 50, 3)
        base, bl, _ = run_fwd(c)
        for t, h in ((5, 0), (lens[0] - 2, Nq - 1)):
            d = dict(c, q=c["q"].clone())
            d["q"][0, t, h] *= factor
            o, lse, _ = run_fwd(d)
            same = torch.ones(lens[0], Nq, dtype=torch.bool, device="cuda")
            same[t, h] = False
            assert torch.equal(o[0][same], base[0][same]) and torch.equal(lse[0][same], bl[0][same]), (Nq, t, h)
            assert not torch.equal(lse[0, t, h], bl[0, t, h])
    c = attn_case(dtype, [1] * 3, 16, 1, 64, 64, 3000, 3, past=[5, 700, 4000], batch=True)
    lens = torch.tensor(c["past"], dtype=torch.int32).cuda()
    step = lambda q: gdr.window_attn_step(q[:, 0].cuda(), dev(c["k"])[:, 0], dev(c["v"])[:, 0], tuple(x.cuda() for x in c["cache"]),
                                          lens, 3000, 3, scale=c["scale"])
    base = step(c["q"])
    for n, h in ((0, 15), (1, 0), (2, 9)):
        q = c["q"].clone()
        q[n, 0, h] *= factor
        o = step(q)
        same = torch.ones(3, 16, dtype=torch.bool, device="cuda")
        same[n, h] = False
        assert torch.equal(o[same], base[same]) and not torch.equal(o[n, h], base[n, h]), (n, h)


def exact_case(dtype, lens, Nq, Nk, dk, dv, window, sinks, e, **kw):
    """Rows of q in threes: whole numbers times 2^e, small ones, whole numbers times -2^e."""
    c = attn_case(dtype, lens, Nq, Nk, dk, dv, window, sinks, scale=0.125, **kw)
    gen = torch.Generator().manual_seed(e + 100)
    whole = lambda *s: torch.randint(-2, 3, s, generator=gen).float()
    q = whole(*c["q"].shape) * 2.0 ** e
    q[:, 2::3] *= -1
    q[:, 1::3] = whole(*q[:, 1::3].shape) * 0.01
    c["q"], c["k"] = q.to(T[dtype]), whole(*c["k"].shape).to(T[dtype])
    if c["cache"] is not None:
        c["cache"][0].copy_(torch.where(c["cache"][0].isnan(), c["cache"][0].float(), whole(*c["cache"][0].shape)))
    return c


def softmax(c, q, k, pq, pk, large):
    """seen, P, lse of one head and the relative error of its weights"""
    seen = oa.sees(pq[:, None], pk[None], c["window"], c["sinks"])
    s = np.where(seen, c["scale"] * (q @ k.T), -np.inf)
    top = s.max(1)
    p = np.exp(s - top[:, None])
    big = large[:, None] & (np.abs(top) > 0)[:, None]
    assert ((s == top[:, None]) | (s <= top[:, None] - 512))[big[:, 0]].all()
    l = p.sum(1)
    p /= l[:, None]
    lse = top + np.log(l)
    return seen, p, lse, np.where(big, np.where(p > 0, 40 * U, 0.0), _weight_error(c, q, k, seen, lse))


def expected(c, o=None):
    """(o, lse, bounds) and, given the call's o, {gradient: [value, bound]}"""
    Nq, Nk, dk, dv = c["dims"]
    G, scale, half = Nq // Nk, c["scale"], half_of(c)
    q, d_o = f64(c["q"]).reshape(-1, Nq, dk), f64(c["d_o"]).reshape(-1, Nq, dv)
    large = np.abs(q).max((1, 2)) > 1
    r, rl, eo, el = np.zeros((len(q), Nq, dv)), np.zeros((len(q), Nq)), np.zeros((len(q), Nq, dv)), np.zeros((len(q), Nq))
    out = {x: [np.zeros(s), np.zeros(s)] for x, s in (("dq", q.shape), ("dk", (len(q), Nk, dk)), ("dv", (len(q), Nk, dv)))}
    for n, rows, pq, pk, k, v in sequences(c):
        for h in range(Nq if len(pq) else 0):
            g, a = h // G, q[rows, h]
            seen, p, lse, e = softmax(c, a, k[:, g], pq, pk, large[rows])
            m, worst = seen.sum(1)[:, None], e.max(1)[:, None]
            r[rows, h], rl[rows, h] = p @ v[:, g], lse
            eo[rows, h] = (half + 2 * worst + 2 * (m + 20 + m / 32 * 10) * U) * (p @ np.abs(v[:, g]))
            el[rows, h] = worst[:, 0] + (m[:, 0] * 1.5 + 40) * U + 8 * U * np.abs(lse)
            if o is None:
                continue
            do, vg, og = d_o[rows, h], v[:, g], o[rows, h]
            dp = do @ vg.T - (do * og).sum(1)[:, None]
            M = np.abs(do) @ np.abs(vg).T + (np.abs(do) * np.abs(og)).sum(1)[:, None]
            # lse as it is stored, where the weights are formed from it
            e = e + np.where(np.abs(lse) * np.log2(np.e) > 1024, 0.0, 8 * U * np.abs(lse))[:, None]
            err = p * ((e + half) * np.abs(dp) + (dv + 4) * U * M) * (1 + half)
            ds, adds = p * np.abs(dp), (len(pq) * G + len(pk) + 70) * U
            for name, i, val, bound in (
                    ("dq", h, scale * (p * dp) @ k[:, g], scale * (err + adds * ds) @ np.abs(k[:, g])),
                    ("dk", g, scale * (p * dp).T @ a, scale * (err + adds * ds).T @ np.abs(a)),
                    ("dv", g, p.T @ do, (p * (e + half + adds)).T @ np.abs(do))):
                out[name][0][rows, i] += val
                out[name][1][rows, i] += bound
    return (r, rl, eo, el) if o is None else out


EXACT = {
    "few_rows": dict(dtype="bf16", lens=[70, 1, 33], Nq=2, Nk=1, dk=64, dv=64, window=50, sinks=4),
    "few_rows_f32": dict(dtype="f32", lens=[90, 41], Nq=2, Nk=1, dk=64, dv=128, window=37, sinks=1),
    "runs_of_sinks": dict(dtype="bf16", lens=[620, 60], Nq=4, Nk=2, dk=128, dv=128, window=60, sinks=5),
    "runs_of_sinks_f32": dict(dtype="f32", lens=[620], Nq=2, Nk=1, dk=128, dv=64, window=60, sinks=5),
    "many_rows": dict(dtype="bf16", lens=[500, 41], Nq=64, Nk=8, dk=64, dv=64, window=100, sinks=4),
    "many_rows_f32": dict(dtype="f32", lens=[540], Nq=64, Nk=16, dk=64, dv=64, window=60, sinks=1),
    "odd": dict(dtype="bf16", lens=[150], Nq=3, Nk=1, dk=63, dv=21, window=64, sinks=0, pad=1),
    "odd_f32": dict(dtype="f32", lens=[130], Nq=3, Nk=1, dk=63, dv=21, window=64, sinks=3, pad=1),
}


@pytest.mark.parametrize("e", [12, 20, 24, 30, 60])
@pytest.mark.parametrize("case", sorted(EXACT))
def test_large_scores(case, e):
    """Outputs and gradients of rows whose scores are up to 2^20 ... 2^68, between rows of small ones."""
    c = exact_case(e=e, **EXACT[case])
    o, lse, _ = run_fwd(c)
    r, rl, eo, el = expected(c)
    within("%s 2^%d o" % (case, e), o, r, eo)
    within("%s 2^%d lse" % (case, e), lse, rl, el)
    for kind in (None, c["q"].dtype):
        got = run_bwd(c, o, lse, grad_dtype=kind)
        ref = expected(c, f64(o).reshape(r.shape))
        for x in ("dq", "dk", "dv"):
            within("%s 2^%d %s" % (case, e, x), got[x], *ref[x])


@pytest.mark.parametrize("e", [12, 24, 60])
@pytest.mark.parametrize("dtype,window", [("bf16", 50), ("f32", 50), ("bf16", 2500), ("f32", 2500)])
def test_large_scores_of_single_tokens_and_pieces(dtype, window, e):
    for lens in ([1] * 4, [40, 3, 70, 1]):
        c = exact_case(dtype, lens, 4, 2, 64, 64, window, 4, e, past=[0, 30, 700, 3000], batch=lens == [1] * 4)
        r, rl, eo, el = expected(c)
        if lens == [1] * 4:
            o = gdr.window_attn_step(*(dev(c[x])[:, 0] for x in "qkv"), tuple(x.cuda() for x in c["cache"]),
                                     torch.tensor(c["past"], dtype=torch.int32).cuda(), window, 4, scale=c["scale"])
        else:
            o, lse, _ = run_fwd(c)
            within("2^%d lse" % e, lse, rl, el)
        within("2^%d o" % e, o, r, eo)


def test_rows_of_infinite_lse():
    """Rows whose scores are all -inf, or one of them +inf, give NaN; the gradients of their sequence may, no others."""
    c = attn_case("f32", [60, 50, 40], 2, 1, 64, 64, 20, 2, seed=3)
    o, lse, _ = run_fwd(c)
    base = run_bwd(c, o, lse)
    c["q"] = c["q"].clone()
    c["q"][0, 70] = 0
    c["q"][0, 70, 0, 0] = 3e38
    c["k"] = c["k"].clone()
    c["k"][0, 60:110, 0, 0] = -1e10
    o2, l2, _ = run_fwd(c)
    assert torch.isnan(o2[0, 70, 0]).all() and torch.isfinite(o2[0, :60]).all() and torch.isfinite(o2[0, 110:]).all()
    got = run_bwd(c, o2, l2)
    for x in ("dq", "dk", "dv"):
        for s in (slice(0, 60), slice(110, None)):
            assert torch.equal(got[x][0, s], base[x][0, s])
    assert torch.isnan(got["dq"][0, 70, 0]).all()
