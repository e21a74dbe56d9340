"""Window attention on the GPU where workgroups share a row's keys: long windows over few rows, parts that hold no key,
and sinks, windows and groups at their ends, against oracle/attn.py within the bounds of tests/attn_common.py."""
import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from attn_common import attn_case, backward_reference, forward_reference, within
from mixer_common import f64, randn
from test_gpu_attn import dev, lens_of, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

FWD = {
    "few_rows": dict(dtype="bf16", lens=[5], past=[9500], Nq=2, Nk=1, dk=64, dv=64, window=9000, sinks=2),
    "few_rows_f32": dict(dtype="f32", lens=[7, 1], past=[5100, 4000], Nq=2, Nk=2, dk=40, dv=72, window=5000, sinks=3),
    "most_parts_empty": dict(dtype="bf16", lens=[20, 3], past=[0, 40], Nq=4, Nk=1, dk=128, dv=128, window=20000, sinks=0),
    "most_parts_empty_f32": dict(dtype="f32", lens=[33], past=None, Nq=1, Nk=1, dk=64, dv=64, window=1 << 30, sinks=9),
    "sinks_shared": dict(dtype="bf16", lens=[40], past=[9000], Nq=2, Nk=1, dk=64, dv=32, window=16, sinks=8500),
    "ring_turned": dict(dtype="bf16", lens=[31, 31], past=[8191, 8250], Nq=2, Nk=1, dk=64, dv=64, window=8192, sinks=1, batch=True),
    "many_rows_f32": dict(dtype="f32", lens=[3001], past=None, Nq=6, Nk=2, dk=64, dv=64, window=2000, sinks=2),
    "odd": dict(dtype="bf16", lens=[9], past=[8300], Nq=3, Nk=1, dk=21, dv=11, window=8200, sinks=5, pad=3),
}


@pytest.mark.parametrize("case", sorted(FWD))
def test_fwd(case):
    c = attn_case(**FWD[case])
    o, lse, eo, el, caches = forward_reference(c)
    got, gl, cache = run_fwd(c)
    within(case + " o", got, o, eo)
    within(case + " lse", gl, lse, el)
    for x, y in zip(cache or (), caches or ()):
        assert np.array_equal(f64(x), y, equal_nan=True)
    again, al, _ = run_fwd(c)
    assert torch.equal(got, again) and torch.equal(gl, al)


STEP = {
    "shared": dict(dtype="bf16", past=[9000, 2], Nq=8, Nk=2, dk=128, dv=128, window=5000, sinks=4),
    "shared_f32": dict(dtype="f32", past=[2500, 4200, 0], Nq=4, Nk=2, dk=72, dv=40, window=2300, sinks=1),
    "parts_empty": dict(dtype="bf16", past=[0, 1, 300, 16000], Nq=2, Nk=1, dk=64, dv=64, window=16384, sinks=0),
    "sinks_shared": dict(dtype="bf16", past=[7000, 3], Nq=2, Nk=1, dk=64, dv=64, window=3, sinks=6000),
    "odd": dict(dtype="bf16", past=[5000, 77], Nq=3, Nk=1, dk=19, dv=33, window=4097, sinks=7, pad=1),
    "forty_heads_of_one": dict(dtype="bf16", past=[3000], Nq=40, Nk=1, dk=64, dv=64, window=4000, sinks=2),
}


@pytest.mark.parametrize("case", sorted(STEP))
def test_step(case):
    kw = dict(STEP[case])
    c = attn_case(lens=[1] * len(kw["past"]), batch=True, **kw)
    o, _, eo, _, caches = forward_reference(c)
    q, k, v = (dev(c[x])[:, 0] for x in "qkv")
    cache = tuple(x.cuda() for x in c["cache"])
    got = gdr.window_attn_step(q, k, v, cache, lens_of(c), c["window"], c["sinks"], scale=c["scale"])
    within(case, got, o, eo)
    for x, y in zip(cache, caches):
        assert np.array_equal(f64(x), y, equal_nan=True)


BWD = {
    "sinks_far_beyond": dict(dtype="bf16", lens=[100], Nq=2, Nk=1, dk=64, dv=64, window=1, sinks=(1 << 31) - 2),
    "window_far_beyond": dict(dtype="f32", lens=[70, 3], Nq=2, Nk=1, dk=32, dv=32, window=(1 << 31) - 1, sinks=0),
    "one_query_behind_the_window": dict(dtype="bf16", lens=[129, 130, 128], Nq=2, Nk=1, dk=64, dv=64, window=128, sinks=3),
    "runs_of_queries": dict(dtype="bf16", lens=[300, 0, 1100], Nq=2, Nk=1, dk=64, dv=32, window=8, sinks=130),
    "seventy_heads_of_one": dict(dtype="f32", lens=[150, 9], Nq=70, Nk=1, dk=16, dv=24, window=12, sinks=2),
}


@pytest.mark.parametrize("case", sorted(BWD))
def test_bwd(case):
    c = attn_case(**BWD[case])
    o, lse, _ = run_fwd(c)
    ref = backward_reference(c, f64(o).reshape(-1, *o.shape[2:]), f64(lse).reshape(-1, lse.shape[2]))
    got = run_bwd(c, o, lse)
    for x in ("dq", "dk", "dv"):
        within("%s %s" % (case, x), got[x], *ref[x])


def test_shared_rows_in_two_graphs_and_on_two_streams():
    """Calls with workspaces at the same time: two graphs replayed on two streams, each against its own eager result."""
    cs = [attn_case("bf16", [6], 2, 1, 64, 64, 9000, 2, past=[9100], seed=s) for s in (1, 2)]
    todo, graphs, outs, keep = [], [], [], []
    for c in cs:
        q, k, v = (dev(c[x]) for x in "qkv")
        cache, lens = tuple(x.cuda() for x in c["cache"]), lens_of(c)
        f = lambda q=q, k=k, v=v, cache=cache, lens=lens: gdr.window_attn_fwd(q, k, v, 9000, 2, cache=cache, lens=lens)
        before = tuple(x.clone() for x in cache)
        want = f()
        for x, y in zip(cache, before):
            x.copy_(y)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            got = f()
        todo.append((cache, before, want))
        keep.append(f)                                  # a graph reads its inputs at every replay
        graphs.append(g)
        outs.append(got)
    streams = [torch.cuda.Stream() for _ in cs]
    for turn in range(4):
        for cache, before, _ in todo:
            for x, y in zip(cache, before):
                x.copy_(y)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, want), got in zip(todo, outs):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), turn
        randn(torch.Generator().manual_seed(turn), 100).cuda().sum()


def test_lens_out_of_range_stay_in_their_buffers():
    """Results are unspecified, but nothing beside the caches is written and the call returns."""
    W, S, N = 20, 3, 2
    for lens in (2 ** 31 - 1, 2 ** 31 - 70):
        gen = torch.Generator().manual_seed(1)
        whole = [torch.full((N + 2, S + W, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cache = tuple(x[1:-1] for x in whole)
        past = torch.full((N,), lens, dtype=torch.int32, device="cuda")
        new = lambda *s: randn(gen, *s, dtype=torch.bfloat16).cuda()
        gdr.window_attn_step(new(N, 4, 64), new(N, 2, 64), new(N, 2, 64), cache, past, W, S)
        gdr.window_attn_fwd(new(N, 40, 4, 64), new(N, 40, 2, 64), new(N, 40, 2, 64), W, S, cache=cache, lens=past)
        for x in whole:
            assert (x[0] == 7).all() and (x[-1] == 7).all()


def test_caches_of_two_billion_tokens():
    """A window of 2^31 - 66 tokens of one element: one key far above the others, at the end of the cache, gives its value."""
    W, past, at = 2 ** 31 - 66, 2 ** 31 - 80, 2 ** 31 - 83
    cache = tuple(torch.zeros(1, W, 1, 1, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache[0][0, at], cache[1][0, at] = 100.0, 5.0
    lens = torch.tensor([past], dtype=torch.int32, device="cuda")
    one = torch.ones(1, 1, 1, dtype=torch.bfloat16, device="cuda")
    assert float(gdr.window_attn_step(one, 0 * one, 2 * one, cache, lens, W, scale=1.0)) == 5.0
    assert float(cache[1][0, past]) == 2.0 and float(cache[1][0, past - 1]) == 0.0
    o, lse = gdr.window_attn_fwd(*(x * torch.ones(1, 3, 1, 1, dtype=torch.bfloat16, device="cuda") for x in (1, 0, 2)), W,
                                 scale=1.0, cache=cache, lens=lens)
    assert (o == 5).all() and ((lse - 100).abs() < 1e-4).all()
    assert (cache[1][0, past:past + 3] == 2).all()
