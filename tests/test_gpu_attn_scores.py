"""Window attention on the GPU where scores are large or infinite: what a token's scores may change, and values."""
import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from attn_common import attn_case
from test_gpu_attn import dev, run_fwd

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
