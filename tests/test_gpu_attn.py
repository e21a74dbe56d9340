"""Window attention on the GPU against oracle/attn.py (float64), within the bounds that tests/attn_common.py derives."""
import ctypes

import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from attn_common import attn_case, backward_reference, forward_reference, within
from chunkwise_gated_delta_local_amd import api
from mixer_common import f64, randn

pytestmark = pytest.mark.gpu


def dev(t):
    return None if t is None else t.cuda()


def lens_of(c):
    return torch.tensor(c["past"], dtype=torch.int32).cuda()


def run_fwd(c, **kw):
    cache = None if c["cache"] is None else tuple(x.cuda() for x in c["cache"])
    o, lse = gdr.window_attn_fwd(dev(c["q"]), dev(c["k"]), dev(c["v"]), c["window"], c["sinks"], scale=c["scale"],
                                 cache=cache, lens=None if cache is None else lens_of(c), cu_seqlens=dev(c["cu"]),
                                 cu_seqlens_cpu=c["cu"], **kw)
    return o, lse, cache


def run_bwd(c, o, lse, **kw):
    return gdr.window_attn_bwd(dev(c["q"]), dev(c["k"]), dev(c["v"]), o, lse, dev(c["d_o"]), c["window"], c["sinks"],
                               scale=c["scale"], cu_seqlens=dev(c["cu"]), cu_seqlens_cpu=c["cu"], **kw)


# name: dtype, lengths, Nq, Nk, dk, dv, window, sinks
CASES = {
    "one_token": dict(dtype="bf16", lens=[1], Nq=1, Nk=1, dk=64, dv=64, window=1, sinks=0),
    "itself_alone": dict(dtype="f32", lens=[70], Nq=2, Nk=1, dk=64, dv=64, window=1, sinks=0),
    "packed": dict(dtype="bf16", lens=[1, 0, 200, 33, 129, 0, 31, 2], Nq=4, Nk=2, dk=128, dv=128, window=50, sinks=4),
    "packed_f32": dict(dtype="f32", lens=[130, 5, 0, 64, 1], Nq=6, Nk=2, dk=72, dv=40, window=37, sinks=1),
    "batch_of_three_heads_each": dict(dtype="bf16", lens=[150] * 3, Nq=6, Nk=2, dk=80, dv=96, window=64, sinks=0, batch=True),
    "tile_edges": dict(dtype="bf16", lens=[64, 65, 63, 128, 32], Nq=2, Nk=2, dk=64, dv=64, window=32, sinks=32),
    "window_behind_all": dict(dtype="bf16", lens=[300], Nq=3, Nk=1, dk=32, dv=128, window=1000, sinks=5),
    "sinks_behind_all": dict(dtype="f32", lens=[90, 20], Nq=2, Nk=1, dk=128, dv=128, window=3, sinks=200),
    "many_sinks": dict(dtype="bf16", lens=[700], Nq=2, Nk=1, dk=64, dv=64, window=65, sinks=150),
    "sinks_f32": dict(dtype="f32", lens=[620, 333], Nq=2, Nk=1, dk=64, dv=128, window=33, sinks=7),
    "odd_dims": dict(dtype="bf16", lens=[75, 20], Nq=5, Nk=1, dk=7, dv=9, window=20, sinks=3),
    "one_dim_f32": dict(dtype="f32", lens=[40], Nq=2, Nk=2, dk=1, dv=1, window=11, sinks=0),
    "odd_dims_f32": dict(dtype="f32", lens=[75], Nq=2, Nk=1, dk=33, dv=101, window=20, sinks=2),
    "strided": dict(dtype="bf16", lens=[100, 77], Nq=4, Nk=2, dk=64, dv=64, window=40, sinks=4, pad=64),
    "strided_odd": dict(dtype="bf16", lens=[100], Nq=4, Nk=2, dk=64, dv=32, window=40, sinks=4, pad=5),
    "strided_odd_f32": dict(dtype="f32", lens=[60, 60], Nq=2, Nk=1, dk=64, dv=64, window=40, sinks=4, pad=3, batch=True),
    "seventy_heads_of_one": dict(dtype="bf16", lens=[40, 9], Nq=70, Nk=1, dk=32, dv=32, window=12, sinks=2),
    "high_scores": dict(dtype="bf16", lens=[150], Nq=2, Nk=1, dk=64, dv=64, window=90, sinks=2, qscale=30.0),
    "high_scores_f32": dict(dtype="f32", lens=[150], Nq=2, Nk=1, dk=64, dv=64, window=90, sinks=2, qscale=30.0),
    "long_rows": dict(dtype="bf16", lens=[500, 41], Nq=64, Nk=8, dk=128, dv=128, window=100, sinks=4),
    "long_rows_f32": dict(dtype="f32", lens=[540], Nq=64, Nk=16, dk=64, dv=128, window=129, sinks=1),
    "long_rows_odd": dict(dtype="bf16", lens=[523], Nq=66, Nk=22, dk=36, dv=20, window=75, sinks=70),
}


@pytest.mark.parametrize("case", sorted(CASES))
def test_fwd(case):
    c = attn_case(**CASES[case])
    o, lse, eo, el, _ = forward_reference(c)
    for out in (None, torch.float32):
        got, gl, _ = run_fwd(c, out_dtype=out)
        assert got.dtype == (c["q"].dtype if out is None else out)
        within(case + " o", got, o, eo)
        within(case + " lse", gl, lse, el)


@pytest.mark.parametrize("grad", ["io", "f32"])
@pytest.mark.parametrize("case", sorted(CASES))
def test_bwd(case, grad):
    """From the forward's own o and lse; in the fp32 variant o and d_o are fp32 too."""
    c = attn_case(**CASES[case])
    full = grad == "f32"
    if full:
        c["d_o"] = c["d_o"].float() * 1.001
    o, lse, _ = run_fwd(c, out_dtype=torch.float32 if full else None)
    got = run_bwd(c, o, lse, grad_dtype=None if full else c["q"].dtype)
    Nq, _, _, dv = c["dims"]
    ref = backward_reference(c, f64(o).reshape(-1, Nq, dv), f64(lse).reshape(-1, Nq), rounded_d_o=full)
    for x in ("dq", "dk", "dv"):
        assert got[x].dtype == (torch.float32 if full else c["q"].dtype) and got[x].shape == c[x[1]].shape
        within("%s %s" % (case, x), got[x], *ref[x])


CACHED = {
    "pieces": dict(dtype="bf16", lens=[30, 1, 0, 100, 64, 5], past=[0, 7, 9, 200, 3, 51], Nq=4, Nk=2, dk=64, dv=64, window=50, sinks=4),
    "pieces_f32": dict(dtype="f32", lens=[40, 12], past=[33, 160], Nq=6, Nk=2, dk=72, dv=40, window=37, sinks=1),
    "no_sinks": dict(dtype="bf16", lens=[70, 70, 70], past=[64, 0, 500], Nq=2, Nk=1, dk=128, dv=128, window=64, sinks=0, batch=True),
    "sinks_not_full": dict(dtype="bf16", lens=[3, 30, 9], past=[2, 5, 10], Nq=2, Nk=1, dk=64, dv=64, window=8, sinks=10),
    "longer_than_the_window": dict(dtype="f32", lens=[90, 41], past=[11, 3], Nq=1, Nk=1, dk=32, dv=32, window=16, sinks=3),
    "window_of_one": dict(dtype="bf16", lens=[5, 8], past=[4, 0], Nq=2, Nk=2, dk=64, dv=64, window=1, sinks=2),
    "odd": dict(dtype="bf16", lens=[20, 33], past=[90, 1], Nq=3, Nk=1, dk=13, dv=5, window=29, sinks=3, pad=1),
    "long_rows": dict(dtype="bf16", lens=[260, 300], past=[77, 1000], Nq=64, Nk=8, dk=128, dv=64, window=90, sinks=5),
    "long_rows_f32": dict(dtype="f32", lens=[520], past=[130], Nq=64, Nk=16, dk=64, dv=64, window=60, sinks=70),
}


@pytest.mark.parametrize("case", sorted(CACHED))
def test_fwd_goes_on_from_caches(case):
    """Rows that hold no token are NaN; the caches afterwards are bit for bit those of the definition, NaN included."""
    c = attn_case(**CACHED[case])
    o, lse, eo, el, caches = forward_reference(c)
    got, gl, cache = run_fwd(c)
    within(case + " o", got, o, eo)
    within(case + " lse", gl, lse, el)
    for x, y in zip(cache, caches):
        assert np.array_equal(f64(x), y, equal_nan=True)


def test_fwd_fills_empty_caches_without_lens():
    c = attn_case("bf16", [40, 9], 2, 1, 64, 64, 16, 4, past=[0, 0], seed=5)
    got, _, cache = run_fwd(c)
    again = tuple(x.cuda() for x in c["cache"])
    o, _ = gdr.window_attn_fwd(dev(c["q"]), dev(c["k"]), dev(c["v"]), 16, 4, cache=again, cu_seqlens=dev(c["cu"]))
    assert torch.equal(o, got) and all(torch.equal(a.nan_to_num(7), b.nan_to_num(7)) for a, b in zip(cache, again))


# ---------------------------------------------------------------- single tokens
STEP = {
    "ragged": dict(dtype="bf16", past=[0, 1, 3, 4, 5, 53, 54, 55, 700, 200], Nq=4, Nk=2, dk=128, dv=128, window=50, sinks=4),
    "f32": dict(dtype="f32", past=[0, 30, 64, 1000], Nq=6, Nk=2, dk=72, dv=40, window=37, sinks=1),
    "no_sinks": dict(dtype="bf16", past=[0, 63, 64, 65], Nq=1, Nk=1, dk=64, dv=64, window=64, sinks=0),
    "window_of_one": dict(dtype="f32", past=[0, 1, 9], Nq=2, Nk=1, dk=64, dv=64, window=1, sinks=0),
    "odd": dict(dtype="bf16", past=[100, 7], Nq=5, Nk=1, dk=13, dv=5, window=29, sinks=3, pad=1),
    "strided": dict(dtype="bf16", past=[100, 7, 33], Nq=4, Nk=2, dk=64, dv=64, window=29, sinks=3, pad=32),
    "one_long": dict(dtype="bf16", past=[5000], Nq=16, Nk=4, dk=128, dv=128, window=1500, sinks=4),
    "one_long_f32": dict(dtype="f32", past=[5000], Nq=4, Nk=1, dk=128, dv=128, window=900, sinks=70),
    "forty_heads_of_one": dict(dtype="bf16", past=[300, 10], Nq=40, Nk=1, dk=64, dv=64, window=100, sinks=2),
    "many": dict(dtype="bf16", past=list(range(0, 600, 4)), Nq=4, Nk=4, dk=64, dv=64, window=200, sinks=1),
}


@pytest.mark.parametrize("case", sorted(STEP))
def test_step(case):
    kw = dict(STEP[case])
    c = attn_case(lens=[1] * len(kw["past"]), batch=True, **kw)
    o, _, eo, _, caches = forward_reference(c)
    for out in (None, torch.float32):
        cache = tuple(x.cuda() for x in c["cache"])
        lens = lens_of(c)
        q, k, v = (dev(c[x])[:, 0] for x in "qkv")
        got = gdr.window_attn_step(q, k, v, cache, lens, c["window"], c["sinks"], scale=c["scale"], out_dtype=out)
        within(case, got, o, eo)
        for x, y in zip(cache, caches):
            assert np.array_equal(f64(x), y, equal_nan=True)
        assert lens.tolist() == c["past"]


@pytest.mark.parametrize("dtype,Nq,Nk,window,sinks", [("bf16", 4, 2, 24, 3), ("f32", 2, 2, 10, 0), ("bf16", 8, 1, 40, 50)])
def test_steps_continue_a_prompt(dtype, Nq, Nk, window, sinks):
    """A prompt, a piece and single tokens: the outputs of the whole prompt, each within the bound of the whole."""
    d, n = 64, 75
    c = attn_case(dtype, [n, n], Nq, Nk, d, d, window, sinks, batch=True, seed=9)
    o, _, eo, _, _ = forward_reference(c)
    q, k, v = (dev(c[x]) for x in "qkv")
    cache = tuple(torch.full((2, sinks + window, Nk, d), float("nan"), dtype=q.dtype, device="cuda") for _ in range(2))
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    outs = []
    for a, b in ((0, 30), (30, 51)):
        outs.append(gdr.window_attn_fwd(*(x[:, a:b].contiguous() for x in (q, k, v)), window, sinks, cache=cache, lens=lens)[0])
        lens += b - a
    for t in range(51, n):
        outs.append(gdr.window_attn_step(q[:, t], k[:, t], v[:, t], cache, lens, window, sinks)[:, None])
        lens += 1
    within("pieces", torch.cat(outs, 1), o.reshape(2, n, Nq, d), eo.reshape(2, n, Nq, d))


def test_step_passes_over_negative_lens():
    """Rows of a padded batch: zero outputs and untouched caches; the others as in a call of their own."""
    for window, past in ((20, [5, 0, 90, 33]), (3000, [2900, 17, 4000, 1])):
        c = attn_case("bf16", [1] * 4, 4, 2, 64, 64, window, 2, past=past, batch=True)
        q, k, v = (dev(c[x])[:, 0] for x in "qkv")
        cache, want = (tuple(x.cuda() for x in c["cache"]) for _ in range(2))
        lens = lens_of(c)
        ref = gdr.window_attn_step(q, k, v, want, lens, window, 2)
        skip = torch.tensor([False, True, False, True], device="cuda")
        got = gdr.window_attn_step(q, k, v, cache, torch.where(skip, torch.tensor(-1, dtype=torch.int32, device="cuda"), lens), window, 2)
        assert torch.equal(got[~skip], ref[~skip]) and not got[skip].any()
        for x, y, old in zip(cache, want, c["cache"]):
            assert torch.equal(x[~skip].nan_to_num(7), y[~skip].nan_to_num(7))
            assert torch.equal(x[skip].nan_to_num(7), old.cuda()[skip].nan_to_num(7))


# ---------------------------------------------------------------- Inf and NaN
@pytest.mark.parametrize("Nq", [2, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_token_reaches_those_that_see_it_alone(dtype, value, Nq):
    """v of a token set to NaN or Inf, and k to NaN: all other tokens keep their bits."""
    lens, window, sinks = [150, 380, 40], 50, 3
    c = attn_case(dtype, lens, Nq, 2, 64, 64, window, sinks)
    base, bl, _ = run_fwd(c)
    off = np.concatenate([[0], np.cumsum(lens)])
    for what in ("v", "k") if value != value else ("v",):
        for n, j in ((1, 100), (1, 1), (0, 149), (2, 0)):
            d = dict(c)
            d[what] = c[what].clone()
            d[what][0, off[n] + j, 0, 5] = value
            o, lse, _ = run_fwd(d)
            p = np.arange(lens[n])
            hit = np.zeros(off[-1], bool)
            hit[off[n]:off[n + 1]] = (p >= j) & ((p - j < window) | (j < sinks))
            hit = torch.tensor(hit).cuda()
            G = Nq // 2
            assert torch.equal(o[0, ~hit], base[0, ~hit]) and torch.equal(lse[0, ~hit], bl[0, ~hit])
            assert torch.equal(o[0, :, G:], base[0, :, G:])                 # the other key head's queries
            assert (~torch.isfinite(o[0, hit][:, :G]).all(-1)).all()


def test_sequences_do_not_touch_in_the_backward_pass():
    c = attn_case("bf16", [100, 70, 131], 4, 2, 64, 64, 30, 2)
    o, lse, _ = run_fwd(c)
    base = run_bwd(c, o, lse)
    for x in "qkv":
        c[x] = c[x].clone()
        c[x][0, 100:170] = float("nan")
    c["d_o"][0, 120] = float("inf")
    got = run_bwd(c, o, lse)
    for x in ("dq", "dk", "dv"):
        for s in (slice(0, 100), slice(170, None)):
            assert torch.equal(got[x][0, s], base[x][0, s])


def test_rows_of_infinite_scores():
    """A query whose scores overflow to -inf has no weights: NaN, as the softmax of such a row is; the others keep theirs."""
    c = attn_case("f32", [40], 2, 1, 32, 32, 8, 0)
    base, _, _ = run_fwd(c)
    c["q"][0, 20, 0], c["k"][0] = 3e38, c["k"][0].abs().neg() * 1e10
    o, lse, _ = run_fwd(c)
    assert torch.isnan(o[0, 20, 0]).all() and torch.isfinite(o[0, 21:]).all()
    assert base.shape == o.shape


# ---------------------------------------------------------------- how it is called
def test_same_bits_twice_and_in_any_company():
    """The same call gives the same bits, and a sequence those of a call of its own."""
    lens = [90, 301, 1, 200]
    c = attn_case("bf16", lens, 4, 2, 64, 64, 40, 4)
    o, lse, _ = run_fwd(c)
    g = run_bwd(c, o, lse)
    for _ in range(3):
        o2, l2, _ = run_fwd(c)
        g2 = run_bwd(c, o, lse)
        assert torch.equal(o, o2) and torch.equal(lse, l2) and all(torch.equal(g[x], g2[x]) for x in g)


def test_gradients_against_differences():
    """dL/dx along random directions against differences of the fp32 forward. A difference over a step s carries the
    forward's error twice (1e-6 of |o|, over s) and the third derivative (s^2)."""
    c = attn_case("f32", [60, 25], 4, 2, 32, 32, 13, 2, seed=4)
    o, lse, _ = run_fwd(c)
    got = run_bwd(c, o, lse)
    gen = torch.Generator().manual_seed(1)
    w = f64(c["d_o"])
    for x in "qkv":
        step = randn(gen, *c[x].shape)
        s = 1e-2
        vals = []
        for sign in (1, -1):
            d = dict(c)
            d[x] = c[x] + sign * s * step
            vals.append((f64(run_fwd(d)[0]) * w).sum())
        slope = (vals[0] - vals[1]) / (2 * s)
        along = (f64(got["d" + x]) * f64(step)).sum()
        size = np.sqrt((f64(got["d" + x]) ** 2).sum())
        assert abs(slope - along) <= 2e-3 * size * max(1.0, np.sqrt(step.numel()) / 30), (x, slope, along, size)


def test_captured_steps():
    """Two graphs of decoding steps in which lens is advanced, replayed in turn between eager work, against the oracle's
    caches by eager steps."""
    Nq, Nk, d, window, sinks, N = 8, 2, 64, 700, 4, 3
    gen = torch.Generator().manual_seed(2)
    mk = lambda: tuple(randn(gen, N, sinks + window, Nk, d, dtype=torch.bfloat16).cuda() for _ in range(2))
    caches = [mk(), mk()]
    copies = [tuple(x.clone() for x in c) for c in caches]
    lens = [torch.tensor([700, 3, 2000], dtype=torch.int32).cuda() for _ in range(2)]
    eager_lens = [x.clone() for x in lens]
    q, k, v = (randn(gen, N, h, d, dtype=torch.bfloat16).cuda() for h in (Nq, Nk, Nk))
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = gdr.window_attn_step(q, k, v, caches[i], lens[i], window, sinks)
            lens[i].add_(1)
        graphs.append(g)
        outs.append(o)
    for turn in range(6):
        for x in (q, k, v):
            x.copy_(randn(gen, *x.shape, dtype=torch.bfloat16))
        for i in (0, 1) if turn % 2 else (1, 0):
            graphs[i].replay()
        for i in range(2):
            want = gdr.window_attn_step(q, k, v, copies[i], eager_lens[i], window, sinks)
            eager_lens[i] += 1
            assert torch.equal(outs[i], want), (turn, i)
            assert all(torch.equal(a, b) for a, b in zip(caches[i], copies[i])) and torch.equal(lens[i], eager_lens[i])
        torch.cuda.synchronize()


def test_captured_forward_and_backward():
    c = attn_case("bf16", [400, 90], 8, 2, 64, 64, 100, 4)
    q, k, v, d_o = (dev(c[x]) for x in ("q", "k", "v", "d_o"))
    cu = dev(c["cu"])

    def both():
        o, lse = gdr.window_attn_fwd(q, k, v, 100, 4, cu_seqlens=cu, cu_seqlens_cpu=c["cu"])
        return [o, lse, *gdr.window_attn_bwd(q, k, v, o, lse, d_o, 100, 4, cu_seqlens=cu, cu_seqlens_cpu=c["cu"]).values()]
    both()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = both()
    gen = torch.Generator().manual_seed(3)
    for _ in range(4):
        for x in (q, k, v, d_o):
            x.copy_(randn(gen, *x.shape, dtype=torch.bfloat16))
        g.replay()
        want = both()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        torch.cuda.synchronize()


def test_another_stream():
    c = attn_case("bf16", [300], 8, 2, 64, 64, 100, 4)
    o, lse, _ = run_fwd(c)
    g = run_bwd(c, o, lse)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o2, l2, _ = run_fwd(c)
        g2 = run_bwd(c, o2, l2)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2) and all(torch.equal(g[x], g2[x]) for x in g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_is_written_beside_the_outputs(dtype):
    """Outputs, caches and workspaces between canaries, at addresses that their element alone aligns."""
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    code = api._DTYPES[t]
    lens, (Nq, Nk, dk, dv, W, S) = [70, 0, 333], (6, 2, 40, 72, 50, 3)
    c = attn_case(dtype, lens, Nq, Nk, dk, dv, W, S, past=[9, 2, 0], seed=8)
    lib, n, N = api.load_library(), sum(lens), len(lens)
    bands = []

    def guarded(numel, dt, odd=True):
        e = torch.empty((), dtype=dt).element_size()
        whole = torch.full((numel * e + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
        inner = whole[512 + (e if odd else 0):][:numel * e]
        bands.append((whole, 512 + (e if odd else 0), numel * e))
        return inner
    P = lambda x: None if x is None else ctypes.c_void_p(x.data_ptr())
    q, k, v, d_o, cu = (dev(c[x]) for x in ("q", "k", "v", "d_o", "cu"))
    prob = api.AttnProblem(1, n, Nq * dk, Nk * dk, Nk * dv, N, Nq, Nk, dk, dv, W, S, 0.2, code, code, code, code)
    size = ctypes.c_size_t(0)

    def workspace(fn):
        assert fn(ctypes.byref(prob), ctypes.byref(size)) == 0
        return guarded(size.value, torch.uint8, odd=False) if size.value else None
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    o, lse = guarded(n * Nq * dv, t), guarded(n * Nq, torch.float32)
    kc, vc = guarded(N * (S + W) * Nk * dk, t), guarded(N * (S + W) * Nk * dv, t)
    for x, y in ((kc, c["cache"][0]), (vc, c["cache"][1])):
        x.copy_(y.cuda().reshape(-1).view(torch.uint8))
    ws = workspace(lib.gdr_window_attn_fwd_workspace_size)
    lens_dev = lens_of(c)
    assert lib.gdr_window_attn_fwd(ctypes.byref(prob), P(q), P(k), P(v), P(kc), P(vc), P(lens_dev), P(cu), P(c["cu"]), P(o),
                                   P(lse), P(ws), ctypes.c_size_t(size.value), stream) == 0
    d = dict(c, scale=0.2)
    ro, rl, eo, el, caches = forward_reference(d)
    as_type = lambda x, dt, *s: x.clone().view(dt).reshape(*s)
    within("o", as_type(o, t, n, Nq, dv), ro, eo)
    within("lse", as_type(lse, torch.float32, n, Nq), rl, el)
    assert np.array_equal(f64(as_type(kc, t, N, S + W, Nk, dk)), caches[0], equal_nan=True)
    assert np.array_equal(f64(as_type(vc, t, N, S + W, Nk, dv)), caches[1], equal_nan=True)
    d.update(past=[0] * N, cache=None)
    o0, l0 = gdr.window_attn_fwd(q, k, v, W, S, scale=0.2, cu_seqlens=cu)
    grads = [guarded(x.numel(), t) for x in (q, k, v)]
    ws = workspace(lib.gdr_window_attn_bwd_workspace_size)
    assert lib.gdr_window_attn_bwd(ctypes.byref(prob), P(q), P(k), P(v), P(o0), P(l0), P(d_o), P(cu), P(c["cu"]),
                                   *(P(x) for x in grads), P(ws), ctypes.c_size_t(size.value), stream) == 0
    ref = backward_reference(d, f64(o0).reshape(n, Nq, dv), f64(l0).reshape(n, Nq))
    for x, y, z in zip(grads, (q, k, v), ("dq", "dk", "dv")):
        within(z, as_type(x, t, *y.shape[1:]), *ref[z])
    torch.cuda.synchronize()
    for whole, at, size in bands:
        assert (whole[:at] == 0xA5).all() and (whole[at + size:] == 0xA5).all()


def test_empty_calls():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    o, lse = gdr.window_attn_fwd(z(2, 0, 4, 64), z(2, 0, 2, 64), z(2, 0, 2, 32), 8, 1)
    assert o.shape == (2, 0, 4, 32) and lse.shape == (2, 0, 4)
    g = gdr.window_attn_bwd(z(2, 0, 4, 64), z(2, 0, 2, 64), z(2, 0, 2, 32), o, lse, o, 8, 1)
    assert g["dk"].shape == (2, 0, 2, 64)
    cache = z(0, 9, 2, 64), z(0, 9, 2, 32)
    assert gdr.window_attn_step(z(0, 4, 64), z(0, 2, 64), z(0, 2, 32), cache, z(0, dtype=torch.int32), 8, 1).shape == (0, 4, 32)
    cu = torch.zeros(4, dtype=torch.int32)
    cache = z(3, 9, 2, 64) + 1, z(3, 9, 2, 64) + 1
    o, _ = gdr.window_attn_fwd(z(1, 0, 4, 64), z(1, 0, 2, 64), z(1, 0, 2, 64), 8, 1, cache=cache, cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu)
    assert o.shape == (1, 0, 4, 64) and (cache[0] == 1).all()


def test_elements_past_31_bits():
    """Prompts and caches of more than 2^31 elements: what lies at their end against the same work alone."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)
    n, H, d, tail, W, S = 140000, 128, 128, 300, 40, 4
    q = new(1, n, H, d)
    assert q.numel() > 1 << 31
    k, v = new(1, n, 8, d), new(1, n, 8, d)
    cu = torch.tensor([0, n - tail, n], dtype=torch.int32)
    kw = dict(cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu)
    end = [x[:, n - tail:].contiguous() for x in (q, k, v)]
    o, lse = gdr.window_attn_fwd(q, k, v, W, S, **kw)
    oe, le = gdr.window_attn_fwd(*end, W, S)
    # the tail alone may be shared out among workgroups otherwise: both lie within a few steps of bf16 of each other
    assert (o[0, n - tail:].float() - oe[0].float()).abs().max() <= 2 ** -6 * oe.abs().max()
    assert (lse[0, n - tail:] - le[0]).abs().max() <= 1e-4
    g = gdr.window_attn_bwd(q, k, v, o, lse, o, W, S, grad_dtype=q.dtype, **kw)
    ge = gdr.window_attn_bwd(*end, o[:, n - tail:].contiguous(), lse[:, n - tail:].contiguous(), o[:, n - tail:].contiguous(),
                             W, S, grad_dtype=q.dtype)
    for x in ("dq", "dk", "dv"):
        assert torch.equal(g[x][0, n - tail:], ge[x][0]), x
    del q, k, v, o, lse, g, ge
    N, W, S = 600, 4096, 4
    cache = new(N, W + S, 8, d), new(N, W + S, 8, d)
    assert cache[0].numel() > 1 << 31
    last = tuple(x[-3:].clone() for x in cache)
    lens = torch.full((N,), 5000, dtype=torch.int32, device="cuda")
    q, k, v = new(N, 16, d), new(N, 8, d), new(N, 8, d)
    o = gdr.window_attn_step(q, k, v, cache, lens, W, S)
    oe = gdr.window_attn_step(q[-3:], k[-3:], v[-3:], last, lens[-3:], W, S)
    assert (o[-3:].float() - oe.float()).abs().max() <= 2 ** -6 * oe.abs().max()
    assert torch.equal(cache[0][-3:], last[0]) and torch.equal(cache[1][-3:], last[1])
