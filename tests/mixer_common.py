"""Inputs, float64 references and error bounds of the layer-operator tests.

Bounds. U = 2^-24 is half a step of fp32 relative to the value. Every output is
a sum of products; with each factor off by a relative error e_i and each sum of
n terms adding n U, it is off by at most (sum of the e_i + n U) times the sum of
the products' absolute values M (the same formulas on absolute values). What the
factors carry, in units of U:
  v_exp_f32, v_log_f32, v_rcp_f32   2 (one unit in the last place)
  exp(-|v|) of an argument v        2 |v| + 4 (scaling by log2 e, its rounding, the instruction)
  softplus(v)                       2 |v| + 12
  silu(v), sigmoid(v)               2 |v| + 8
  exp(delta A), per token           |delta A| (20 + error of delta) + 3: A log2 e, the product, for joined
                                    pieces the sum of up to 16 deltas; then the instruction and one update
A stored bf16 value adds half its step, 2^-8 of the value (eps / 2).
"""
import numpy as np
import torch

U = 2.0 ** -24
T = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def close(name, got, ref, M, kappa):
    """|got - ref| <= kappa U M + half a step of got's type."""
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(f64(got).reshape(ref.shape) - ref)
    bound = kappa * U * M * (1 + half) + half * np.abs(ref) + 1e-37
    worst = float(np.max(err / bound)) if err.size else 0.0
    print("%s: worst error / bound %.3f (kappa %.0f)" % (name, worst, kappa), flush=True)
    assert np.isfinite(f64(got)).all(), name
    assert worst <= 1.0, (name, worst, float(err.max()))


def randn(gen, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen) * std + mean).to(dtype)


def strided(t, pad):
    """The same values as a slice of wider tokens (pad more elements each)."""
    if not pad:
        return t
    flat = t.reshape(t.shape[0] * t.shape[1], -1)
    wide = torch.full((flat.shape[0], flat.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :flat.shape[1]] = flat
    st = wide.stride(0)
    inner = [1]
    for n in reversed(t.shape[3:]):
        inner.insert(0, inner[0] * n)
    return wide.as_strided(t.shape, (t.shape[1] * st, st, *inner))


def packed(lens, batch):
    """(lead dims, cu on the CPU or None) for sequences of these lengths, packed or as rows of a batch."""
    if batch:
        assert len(set(lens)) == 1
        return (len(lens), lens[0]), None
    return (1, int(sum(lens))), torch.tensor(offsets(lens), dtype=torch.int32)
