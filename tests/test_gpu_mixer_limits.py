"""The layer operators at the limits of what they take: strides, values, rows, channels."""
import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr

pytestmark = pytest.mark.gpu


def normal(gen, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scan_step_of_time_slices(dtype):
    """One token out of [N, T, ...] tensors whose sequences are 2^22 elements apart and more: the bits of the same token
    alone."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    N, D, G, S = 3, 4096, 2, 16
    x, dt, z = (normal(gen, N, 1100, D, dtype=dtype)[:, t] for t in (0, 7, 1099))
    B, C = (normal(gen, N, 140000, G, S, dtype=dtype)[:, t] for t in (3, 139999))
    assert min(x.stride(0), B.stride(0)) > 1 << 22
    A, D_, bias = -torch.rand(D, S, device="cuda"), normal(gen, D), normal(gen, D)
    h0 = normal(gen, N, D, S)

    def step(f, state):
        return gdr.scan_step(f(x), f(dt), A, f(B), f(C), state, D_, f(z), bias, True), state
    sliced, alone = step(lambda t: t, h0.clone()), step(lambda t: t.contiguous(), h0.clone())
    assert torch.equal(sliced[0], alone[0]) and torch.equal(sliced[1], alone[1])
    assert not torch.equal(alone[1], h0)
