"""Inputs, float64 references and error bounds of the window attention's tests.

Bounds, with U = 2^-24 and half = half a step of the type that weights are rounded to for their products (2^-8 for
bf16 inputs, 0 for fp32). For one query over n keys, Ms = scale sum |q||k| the largest sum of a score's absolute values:
  score                 (dk + 2) U Ms
  weight exp(s - ref)   e = that + (2 |s - ref| + |ref| + 8) U relative: scaling by log2 e, its rounding, v_exp_f32
  sums over n keys      n U relative to the sum of absolute values; each of the n / 32 tiles may also rescale what was
                        summed by a factor of relative error 2 |ref| U + 8 U
  o = sum w v / sum w   (half + 2 e + 2 (n + 20) U) sum p |v|
  lse                   e + (n + 20) U + 4 U |lse|
Backward, with Mg = sum |d_o||v| and Md = sum |d_o||o| (a d_o in fp32 is rounded to the io type first: another half of
each) and lse itself carrying 2 U |lse| when it is scaled:
  dS = P (dP - delta)   P ((e + half) |dP - delta| + ((dv + 2) U + half') (Mg + Md)),  half' = half for a rounded d_o
  dq, dk                scale times the sums of that times |k| or |q|, n U of the sum for adding
  dv                    sum P |d_o| (e + half + half' + n U)
"""
import numpy as np
import torch

from mixer_common import T, U, f64, offsets, packed, randn, strided
from oracle import attn as oa

GARBAGE = float("nan")


def attn_case(dtype, lens, Nq, Nk, dk, dv, window, sinks, past=None, batch=False, pad=0, scale=None, seed=0, qscale=1.0):
    """Inputs on the CPU. past: tokens behind each sequence; its caches then hold what those left, and NaN where no
    token lies."""
    gen = torch.Generator().manual_seed(seed)
    lead, cu = packed(lens, batch)
    t, N = T[dtype], len(lens)
    c = dict(q=strided(randn(gen, *lead, Nq, dk, dtype=t, std=qscale), pad), k=strided(randn(gen, *lead, Nk, dk, dtype=t), pad),
             v=strided(randn(gen, *lead, Nk, dv, dtype=t), pad), d_o=randn(gen, *lead, Nq, dv, dtype=t), cu=cu,
             lens=list(lens), window=window, sinks=sinks, scale=dk ** -0.5 if scale is None else scale,
             past=[0] * N if past is None else list(past), cache=None, dims=(Nq, Nk, dk, dv))
    if past is not None:
        kc, vc = torch.full((N, sinks + window, Nk, dk), GARBAGE).to(t), torch.full((N, sinks + window, Nk, dv), GARBAGE).to(t)
        for n, p in enumerate(past):
            for pos in oa.cached_positions(p, window, sinks):
                kc[n, oa.slot(pos, window, sinks)] = randn(gen, Nk, dk, dtype=t)
                vc[n, oa.slot(pos, window, sinks)] = randn(gen, Nk, dv, dtype=t)
        c["cache"] = (kc, vc)
    return c


def sequences(c):
    """(n, rows of the tokens, positions of queries, positions of keys, k, v) with the cached keys in front."""
    Nq, Nk, dk, dv = c["dims"]
    off = offsets(c["lens"])
    k, v = f64(c["k"]).reshape(-1, Nk, dk), f64(c["v"]).reshape(-1, Nk, dv)
    for n, (a, b) in enumerate(zip(off[:-1], off[1:])):
        past = c["past"][n]
        old = oa.cached_positions(past, c["window"], c["sinks"])
        new = list(range(past, past + b - a))
        kk, vv = k[a:b], v[a:b]
        if old:
            at = [oa.slot(p, c["window"], c["sinks"]) for p in old]
            kk = np.concatenate([f64(c["cache"][0][n, at]), kk])
            vv = np.concatenate([f64(c["cache"][1][n, at]), vv])
        yield n, slice(a, b), np.array(new, dtype=np.int64), np.array(old + new, dtype=np.int64), kk, vv


def half_of(c):
    return torch.finfo(torch.bfloat16).eps / 2 if c["q"].dtype == torch.bfloat16 else 0.0


def _weight_error(c, q, k, seen, ref):
    """e of every weight: [n, m]"""
    scale, dk = c["scale"], q.shape[1]
    s = scale * (q @ k.T)
    Ms = scale * (np.abs(q) @ np.abs(k).T)
    # the running reference lies between the lowest and the highest score that are seen
    top = np.where(seen, np.abs(s), 0.0).max(1, initial=0.0)[:, None]
    return np.where(seen, ((dk + 2) * Ms + 2 * np.abs(s - ref[:, None]) + 3 * top + 2 * np.abs(ref)[:, None] + 30) * U, 0.0)


def forward_reference(c):
    """o [tokens, Nq, dv], lse [tokens, Nq], their bounds, and the caches after the call."""
    Nq, Nk, dk, dv = c["dims"]
    G, W, S = Nq // Nk, c["window"], c["sinks"]
    q = f64(c["q"]).reshape(-1, Nq, dk)
    n_all = len(q)
    o, lse, eo, el = np.zeros((n_all, Nq, dv)), np.zeros((n_all, Nq)), np.zeros((n_all, Nq, dv)), np.zeros((n_all, Nq))
    caches = None if c["cache"] is None else [f64(x).copy() for x in c["cache"]]
    for n, rows, pq, pk, k, v in sequences(c):
        if len(pq) == 0:
            continue
        seen = oa.sees(pq[:, None], pk[None], W, S)
        for h in range(Nq):
            g = h // G
            o[rows, h], lse[rows, h], p = oa.attend(q[rows, h], k[:, g], v[:, g], pq, pk, W, S, c["scale"])
            e = _weight_error(c, q[rows, h], k[:, g], seen, lse[rows, h])
            m = seen.sum(1)[:, None]
            worst = e.max(1)[:, None]
            # a tile may rescale the sums: 1 / 32 of the tiles' keys, 10 U and the score's range each
            eo[rows, h] = (half_of(c) + 2 * worst + 2 * (m + 20 + m / 32 * 10) * U) * (p @ np.abs(v[:, g]))
            el[rows, h] = worst[:, 0] + (m[:, 0] * 1.5 + 30) * U + 4 * U * np.abs(lse[rows, h])
        if caches is not None:
            off, past = rows.start, c["past"][n]
            for i, x in enumerate((c["k"], c["v"])):
                flat = f64(x).reshape((-1,) + x.shape[-2:])
                caches[i][n] = oa.keep(caches[i][n], flat[off:rows.stop], past, W, S)
    return o, lse, eo, el, caches


def backward_reference(c, o, lse, rounded_d_o=False):
    """dict of (gradient, bound), for o and lse as the call gets them (float64 arrays)."""
    Nq, Nk, dk, dv = c["dims"]
    G, W, S, scale, half = Nq // Nk, c["window"], c["sinks"], c["scale"], half_of(c)
    q, d_o = f64(c["q"]).reshape(-1, Nq, dk), f64(c["d_o"]).reshape(-1, Nq, dv)
    more = half if rounded_d_o else 0.0
    out = {x: [np.zeros(s), np.zeros(s)] for x, s in (("dq", q.shape), ("dk", (len(q), Nk, dk)), ("dv", (len(q), Nk, dv)))}
    for n, rows, pq, pk, k, v in sequences(c):
        if len(pq) == 0:
            continue
        seen = oa.sees(pq[:, None], pk[None], W, S)
        for h in range(Nq):
            g = h // G
            a = (q[rows, h], k[:, g], v[:, g], o[rows, h], lse[rows, h], d_o[rows, h])
            for name, x in zip(("dq", "dk", "dv"), oa.attend_backward(*a, pq, pk, W, S, scale)):
                out[name][0][rows, h if name == "dq" else g] += x
            p = np.where(seen, np.exp(np.where(seen, scale * (a[0] @ a[1].T), 0.0) - a[4][:, None]), 0.0)
            e = _weight_error(c, a[0], a[1], seen, a[4])
            dp = a[5] @ a[2].T - (a[5] * a[3]).sum(1)[:, None]
            M = np.abs(a[5]) @ np.abs(a[2]).T + (np.abs(a[5]) * np.abs(a[3])).sum(1)[:, None]
            err = p * ((e + half) * np.abs(dp) + ((dv + 4) * U + more) * M) * (1 + half)
            ds = p * np.abs(dp)
            adds = (len(pk) + 10) * U
            out["dq"][1][rows, h] += scale * ((err + adds * ds) @ np.abs(a[1]))
            adds = (len(pq) * G + 60) * U
            out["dk"][1][rows, g] += scale * ((err + adds * ds).T @ np.abs(a[0]))
            out["dv"][1][rows, g] += (p * (e + half + more + adds)).T @ np.abs(a[5])
    return out


def within(name, got, ref, bound):
    """|got - ref| <= bound + half a step of got's type, element by element."""
    half = torch.finfo(got.dtype).eps / 2
    x = f64(got).reshape(ref.shape)
    assert np.isfinite(x).all(), name
    limit = bound * (1 + half) + half * np.abs(ref) + 1e-37
    worst = float((np.abs(x - ref) / limit).max()) if x.size else 0.0
    print("%s: worst error / bound %.3f" % (name, worst), flush=True)
    assert worst <= 1.0, (name, worst)
