"""Window attention on the GPU: what a sequence's results depend on. Gradients are bit for bit those of the sequence alone;
the forward pass, which shares rows out by the whole call, stays within its bounds in any company; a query without
weights leaves all others as they are."""
import numpy as np
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from attn_common import attn_case, forward_reference, within
from test_gpu_attn import dev, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

CASES = {
    "runs_of_sinks": dict(dtype="bf16", lens=[90, 301, 1, 0, 2900, 200, 17], Nq=4, Nk=2, dk=64, dv=64, window=40, sinks=4),
    "runs_of_sinks_f32": dict(dtype="f32", lens=[1300, 33, 0, 700], Nq=2, Nk=1, dk=128, dv=64, window=100, sinks=9),
    "more_sinks_than_tokens": dict(dtype="bf16", lens=[40, 700, 150, 151], Nq=2, Nk=1, dk=128, dv=128, window=30, sinks=150),
    "window_of_the_longest": dict(dtype="bf16", lens=[100, 1500, 699, 700, 701], Nq=8, Nk=2, dk=64, dv=128, window=700, sinks=2),
    "many_heads": dict(dtype="bf16", lens=[130, 1, 64, 500], Nq=64, Nk=8, dk=64, dv=64, window=64, sinks=3),
    "odd": dict(dtype="f32", lens=[75, 400], Nq=3, Nk=1, dk=33, dv=21, window=50, sinks=1),
    "far": dict(dtype="bf16", lens=[90, 700, 33], Nq=4, Nk=2, dk=64, dv=64, window=40, sinks=4, qscale=3000.0),
}


@pytest.mark.parametrize("batch", [False, True])
@pytest.mark.parametrize("case", sorted(CASES))
def test_gradients_are_those_of_the_sequence_alone(case, batch):
    kw = dict(CASES[case])
    if batch:
        kw["lens"] = [sorted(kw["lens"])[-2]] * 3
    c = attn_case(batch=batch, **kw)
    o, lse, _ = run_fwd(c)
    f32 = c["q"].dtype == torch.float32
    for grad in (None, c["q"].dtype):
        d_o = c["d_o"] if grad or f32 else c["d_o"].float() * 1.001
        g = run_bwd(dict(c, d_o=d_o), o, lse, grad_dtype=grad)
        flat = lambda t: t.reshape((1, -1) + t.shape[2:])
        at = 0
        for n in kw["lens"]:
            cut = lambda t: flat(dev(t))[:, at:at + n].contiguous()
            alone = gdr.window_attn_bwd(cut(c["q"]), cut(c["k"]), cut(c["v"]), cut(o), cut(lse), cut(d_o), c["window"], c["sinks"],
                                        scale=c["scale"], grad_dtype=grad)
            for x in ("dq", "dk", "dv"):
                assert torch.isfinite(alone[x]).all() and torch.equal(flat(g[x])[:, at:at + n], alone[x]), (x, at, n)
            at += n


def test_outputs_stay_within_their_bounds_in_any_company():
    """A sequence by itself, where few rows share their keys, and packed with so many that they do not."""
    lens = [90, 301, 1, 200] + [64] * 80
    c = attn_case("bf16", lens, 8, 1, 64, 64, 40, 4)
    o, lse, eo, el, _ = forward_reference(c)
    got, gl, _ = run_fwd(c)
    within("packed o", got, o, eo)
    within("packed lse", gl, lse, el)
    at = 0
    for n in lens[:5]:
        cut = lambda t: dev(t)[:, at:at + n].contiguous()
        a, b = gdr.window_attn_fwd(cut(c["q"]), cut(c["k"]), cut(c["v"]), 40, 4)
        within("alone o", a, o[at:at + n], eo[at:at + n])
        within("alone lse", b, lse[at:at + n], el[at:at + n])
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq,n", [(4, 40), (64, 600)])
def test_a_query_without_weights_leaves_the_others(dtype, Nq, n):
    """One head's scores of one token overflow to -inf: its output is NaN; every other output, and all gradients of the
    other key head, keep their bits."""
    c = attn_case(dtype, [n], Nq, 2, 32, 32, 8, 0)
    c["k"] = c["k"].clone()
    c["k"][..., 0] = -4.0
    base, bl, _ = run_fwd(c)
    bg = run_bwd(c, base, bl)
    c["q"] = c["q"].clone()
    c["q"][0, 20, 0] = 0.0
    c["q"][0, 20, 0, 0] = 3e38
    o, lse, _ = run_fwd(c)
    other = torch.ones(n, Nq, dtype=torch.bool, device="cuda")
    other[20, 0] = False
    assert torch.isnan(o[0, 20, 0]).all()
    assert torch.equal(o[0][other], base[0][other]) and torch.equal(lse[0][other], bl[0][other])
    g = run_bwd(c, o, lse)
    assert torch.isnan(g["dq"][0, 20, 0]).all() and torch.equal(g["dq"][0, :, Nq // 2:], bg["dq"][0, :, Nq // 2:])
    for x in ("dk", "dv"):
        assert torch.equal(g[x][0, :, 1], bg[x][0, :, 1])
