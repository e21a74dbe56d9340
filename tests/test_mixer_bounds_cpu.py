"""tests/mixer_bounds.py on the CPU: its references are the oracle's, a token-by-token run in fp32 lies within its bounds,
and mistakes of the size that the segmented scan could make, planted in the oracle's results, do not."""
import numpy as np
import pytest
import torch

from mixer_bounds import excess, scan_bounds
from mixer_common import f64
from oracle import mixer as om
from test_gpu_mixer import SCAN, scan_case

NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "dh0")


def case(name):
    c = scan_case(**SCAN[name])
    n, D = len(c["pre"]), c["ref"]["A"].shape[0]
    dy, dl = f64(c["d_y"]).reshape(n, D), f64(c["dl"])
    ref, err = scan_bounds(c["ref"], c["pre"], c["soft"], c["zf"], dy, dl)
    return c, dy, dl, ref, err


@pytest.mark.parametrize("name", ["packed", "state_7_odd", "segments", "bare"])
def test_references(name):
    c, dy, dl, ref, _ = case(name)
    gate = 1.0 if c["zf"] is None else om.silu(c["zf"])
    v, _, last = om.scan(**c["ref"])
    want = dict(zip(NAMES, om.scan_backward(**c["ref"], ds=dy * gate, d_last=dl)), y=v * gate, last=last)
    if c["soft"]:
        want["ddt"] = want["ddt"] / (1 + np.exp(-c["pre"]))
    for k, w in want.items():
        assert np.allclose(ref[k], w, rtol=1e-12, atol=1e-12), k


@pytest.mark.parametrize("name", ["segments", "segments_state_64", "bare"])
def test_fp32_run_lies_within(name):
    c, _, _, ref, err = case(name)
    r = {k: v if k == "cu" else v.astype(np.float32) for k, v in c["ref"].items()}
    A2 = r["A"] * np.float32(1.4426950408889634)
    D, last, y = A2.shape[0], r["h0"].copy(), np.zeros_like(r["x"])
    for q in range(len(r["cu"]) - 1):
        for t in range(r["cu"][q], r["cu"][q + 1]):
            a = np.exp2(A2 * r["delta"][t][:, None])
            last[q] = a * last[q] + (r["delta"][t] * r["x"][t])[:, None] * np.repeat(r["B"][t], D // r["B"].shape[1], 0)
            y[t] = (np.repeat(r["C"][t], D // r["C"].shape[1], 0) * last[q]).sum(1, dtype=np.float32) + r["skip"] * r["x"][t]
    if c["zf"] is not None:
        y = y * om.silu(c["zf"]).astype(np.float32)
    assert excess(y, ref["y"], err["y"]) <= 1.0 and excess(last, ref["last"], err["last"]) <= 1.0


@pytest.mark.parametrize("name", ["segments", "segments_groups", "segments_state_64", "segments_bare"])
def test_planted_mistakes_are_seen(name):
    """A cut of the first sequence at a segment's end: its second part from a state held in bf16 or from zero, G likewise
    in reverse, and parameter gradients that lack a segment or are zero."""
    c, dy, dl, ref, err = case(name)
    r, e = c["ref"], int(c["ref"]["cu"][1])
    cut = 384
    gate = np.ones_like(dy) if c["zf"] is None else om.silu(c["zf"])

    def part(i, j, h0):
        p = {k: r[k][i:j] for k in ("x", "delta", "B", "C")}
        return dict(p, A=r["A"], skip=r["skip"], cu=np.array([0, j - i]), h0=h0)
    ds = dy * gate
    mid = om.scan(**part(0, cut, r["h0"][:1]))[2]
    later = dict(zip(NAMES, om.scan_backward(**part(cut, e, mid), ds=ds[cut:e], d_last=dl[:1])))
    bf16 = lambda a: torch.tensor(a).bfloat16().double().numpy()
    for wrong in (bf16, np.zeros_like):
        v, _, last = om.scan(**part(cut, e, wrong(mid)))
        assert excess(v * gate[cut:e], ref["y"][cut:e], err["y"][cut:e]) > 3
        first = dict(zip(NAMES, om.scan_backward(**part(0, cut, r["h0"][:1]), ds=ds[:cut], d_last=wrong(later["dh0"]))))
        assert excess(first["dx"], ref["dx"][:cut], err["dx"][:cut]) > 3
    first = dict(zip(NAMES, om.scan_backward(**part(0, cut, r["h0"][:1]), ds=ds[:cut], d_last=later["dh0"])))
    for k in ("dA", "dD"):
        assert excess(ref[k] - first[k], ref[k], err[k]) > 3, k      # the first segment's share is missing
        assert excess(np.zeros_like(ref[k]), ref[k], err[k]) > 3, k
    assert excess(ref["ddt_bias"] - ref["ddt"][:cut].sum(0), ref["ddt_bias"], err["ddt_bias"]) > 3
    assert excess(np.zeros_like(ref["ddt_bias"]), ref["ddt_bias"], err["ddt_bias"]) > 3
