"""The selective state space scan, forward and backward, within the bounds that follow an error token by token
(tests/mixer_bounds.py): sequences cut into segments above all."""
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from mixer_bounds import U, check, scan_bounds
from mixer_common import f64
from test_gpu_mixer import SCAN, dev, run_scan, scan_args, scan_case

pytestmark = pytest.mark.gpu

CASES = dict(
    SCAN,
    segments_state_8=dict(dtype="f32", lens=[1030, 5], D=40, S=8),
    segments_state_30=dict(dtype="bf16", lens=[900, 513], D=17, S=30),
    segments_even=dict(dtype="bf16", lens=[1024, 1024, 1024], D=48, S=16, batch=True, pad=4),
    segments_long=dict(dtype="f32", lens=[4000], D=5, S=3),
)
# the bound's median relative to the outputs' size: sums over thousands of tokens are bounded less tightly
MOST = dict(dA=5e-3, dD=1e-2, ddt_bias=3e-2)


@pytest.mark.parametrize("dy", ["io", "f32"])
@pytest.mark.parametrize("case", sorted(CASES))
def test_scan(case, dy):
    """fp32 outputs and gradients; d_y in the io type or in fp32."""
    c = scan_case(**CASES[case])
    n, D = len(c["pre"]), c["ref"]["A"].shape[0]
    if dy == "f32":
        c["d_y"] = c["d_y"].float() + torch.randn(c["d_y"].shape, generator=torch.Generator().manual_seed(9)) / 1024
    ref, err = scan_bounds(c["ref"], c["pre"], c["soft"], c["zf"], f64(c["d_y"]).reshape(n, D), f64(c["dl"]))
    y, last = run_scan(c, out_dtype=torch.float32)
    got = dict(run_scan(c, back=True), y=y, last=last)
    assert set(got) == set(ref)
    for k in ref:
        check("%s %s" % (case, k), got[k], ref[k], err[k], MOST.get(k, 3e-4))


@pytest.mark.parametrize("case", ["segments", "segments_state_8", "segments_state_64", "segments_long"])
def test_segments_against_consecutive_calls(case):
    """One call against calls of at most 500 tokens each, which are not cut: states handed on, gradients handed back."""
    c = scan_case(**CASES[case])
    n, D = len(c["pre"]), c["ref"]["A"].shape[0]
    _, err = scan_bounds(c["ref"], c["pre"], c["soft"], c["zf"], f64(c["d_y"]).reshape(n, D), f64(c["dl"]))
    whole = dict(zip(("y", "last"), run_scan(c, out_dtype=torch.float32)), **run_scan(c, back=True))
    a, k = scan_args(c)
    d_y, dl, h0, cu = dev(c["d_y"]), dev(c["dl"]), dev(c["h0"]), c["ref"]["cu"]
    total = {g: torch.zeros_like(whole[g], dtype=torch.float64) for g in ("dA", "dD", "ddt_bias")}

    def cut(q, i, j):
        s = lambda t: t[:, i:j].contiguous()
        return [s(a[0]), s(a[1]), a[2], s(a[3]), s(a[4])], dict(k, z=None if k["z"] is None else s(k["z"]))

    def close(name, got, at):
        # each side is off by the bound
        bound = 2 * 1.02 * U * torch.tensor(err[name][at], device="cuda").reshape(got.shape) + 1e-37
        assert bool(((whole[name].reshape(err[name].shape)[at].reshape(got.shape).double() - got.double()).abs() <= bound).all()), name
    for q in range(len(cu) - 1):
        ends = sorted({int(cu[q + 1]), *range(int(cu[q]), int(cu[q + 1]), 500)})
        state, parts = h0[q:q + 1], list(zip(ends, ends[1:]))
        entry = []
        for i, j in parts:
            entry.append(state)
            x, kw = cut(q, i, j)
            y, state = gdr.scan_fwd(*x, initial_state=state, out_dtype=torch.float32, **kw)
            close("y", y, slice(i, j))
        close("last", state, slice(q, q + 1))
        G = dl[q:q + 1].contiguous()
        for (i, j), st in reversed(list(zip(parts, entry))):
            x, kw = cut(q, i, j)
            g = gdr.scan_bwd(*x, d_y[:, i:j].contiguous(), initial_state=st, d_final_state=G, **kw)
            for name in ("dx", "ddt", "dB", "dC", "dz"):
                if name in g:
                    close(name, g[name], slice(i, j))
            for name in total:
                total[name] += g[name].double()
            G = g["dh0"]
        close("dh0", G, slice(q, q + 1))
    for name, t in total.items():
        close(name, t, slice(None))
        assert float(t.abs().max()) > 0
