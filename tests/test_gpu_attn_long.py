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
