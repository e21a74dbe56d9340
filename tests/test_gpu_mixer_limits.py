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


@pytest.mark.parametrize("S", [16, 6])
def test_transitions_that_forget_at_once_in_one_token(S):
    """A = -inf and A near the lowest float, step sizes of zero among them (softplus far below its underflow, or dt = 0):
    a token alone leaves the state that a prompt of one token leaves, bit for bit: exp(-inf 0) counts as 1."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    N, D = 5, 48
    x, z = normal(gen, N, D), normal(gen, N, D)
    B, C, h0 = normal(gen, N, 1, S), normal(gen, N, 1, S), normal(gen, N, D, S)
    A = -torch.rand(D, S, device="cuda")
    A[1], A[:, 3], A[7, 2] = float("-inf"), float("-inf"), -3e38
    for soft, dt, zero in ((True, normal(gen, N, D), -300.0), (False, torch.rand(N, D, device="cuda"), 0.0)):
        dt[1], dt[3, ::2] = zero, zero
        state = h0.clone()
        y = gdr.scan_step(x, dt, A, B, C, state, z=z, dt_softplus=soft)
        one = lambda t: t[:, None].contiguous()
        yp, last = gdr.scan_fwd(one(x), one(dt), A, one(B), one(C), z=one(z), dt_softplus=soft, initial_state=h0)
        assert torch.isfinite(state).all() and torch.isfinite(y).all()
        assert torch.equal(state, last)
        assert torch.equal(state[1], h0[1])                 # no step: the state stays
        # two orders of a sum of S products and the gate
        bound = (S + 4) * 2.0 ** -24 * ((C.abs() * last.abs()).sum(-1) * z.abs()) + 1e-30
        assert ((y - yp[:, 0]).abs() <= 2 * bound).all()


def test_norm_of_more_rows_than_threads_of_a_launch():
    """2^30 + 37 short rows, forward and backward: the bits of the same rows in smaller calls."""
    rows, cols, part = (1 << 30) + 37, 2, 1 << 28
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(0, 1 << 14, (rows, cols), generator=gen, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    w, b = normal(gen, cols), normal(gen, cols)
    y, mean, rstd = gdr.layer_norm_fwd(x, w, b)
    dx = gdr.layer_norm_bwd(x, y, mean, rstd, w, grad_dtype=x.dtype)["dx"]
    for i in range(0, rows, part):
        s = slice(i, min(i + part, rows))
        ys, ms, rs = gdr.layer_norm_fwd(x[s], w, b)
        assert torch.equal(y[s], ys) and torch.equal(mean[s], ms) and torch.equal(rstd[s], rs), i
        assert torch.equal(dx[s], gdr.layer_norm_bwd(x[s], ys, ms, rs, w, grad_dtype=x.dtype)["dx"]), i
    assert float(rstd.max()) <= 1e-5 ** -0.5 * 1.001 and bool((mean[-37:] > 0).any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,G,S", [(40, 2, 16), (19, 1, 5), (16, 1, 40)])
def test_scan_of_the_widest_rows(dtype, D, G, S):
    """Tokens 2^22 - 1 elements apart, the most that the tiles' 31-bit offsets take, with channels that leave lanes idle:
    the bits of dense inputs, forward and backward."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    T, width = 300, (1 << 22) - 1
    wide = torch.empty(1, T, width, device="cuda", dtype=dtype)
    ends = (0, D, width - D)                                # slices at both ends of a row
    x, dt, z = (wide[..., i:i + D] for i in ends)
    B, C = (wide[..., i:i + G * S].unflatten(-1, (G, S)) for i in (2 * D, width // 2))
    for t in (x, dt, z, B, C):
        t.copy_(normal(gen, *t.shape, dtype=dtype))
    A, h0 = -torch.rand(D, S, device="cuda"), normal(gen, 1, D, S)
    d_y = normal(gen, 1, T, D, dtype=dtype)

    def all_of(f):
        a = [f(x), f(dt), A, f(B), f(C)]
        kw = dict(z=f(z), dt_softplus=True, initial_state=h0)
        return [*gdr.scan_fwd(*a, **kw), *gdr.scan_bwd(*a, d_y, grad_dtype=dtype, **kw).values()]
    for i, (a, b) in enumerate(zip(all_of(lambda t: t), all_of(lambda t: t.contiguous()))):
        assert torch.isfinite(a).all() and torch.equal(a, b), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bases_aligned_to_an_element_only(dtype):
    """Every tensor one element behind an aligned address: the bits of aligned ones."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    N, T, D, G, S = 2, 70, 72, 2, 16

    def odd(t):
        buf = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)
        out = buf[1:].view(t.shape)
        assert out.data_ptr() % 16 and out.is_contiguous()
        return out.copy_(t)
    io = lambda *s: normal(gen, *s, dtype=dtype)
    x, dt, z, d_y, B, C = io(N, T, D), io(N, T, D), io(N, T, D), io(N, T, D), io(N, T, G, S), io(N, T, G, S)
    f32 = [normal(gen, *s) for s in ((D, 4), (D, 3), (D,), (D, S), (N, D, S))]
    w4, w3, b, A, h0 = f32[0], f32[1], f32[2], -f32[3].abs(), f32[4]
    rows = io(N, 3, D)

    def all_of(f):
        out = []
        for w, r in ((f(w4), f(rows)), (f(w3), f(rows[:, :2].contiguous()))):
            out += gdr.conv_fwd(f(x), w, f(b), initial_state=r)
            out += gdr.conv_bwd(f(x), w, f(d_y), f(b), initial_state=r, d_final_state=r, grad_dtype=dtype).values()
            out += [gdr.conv_step(f(x[:, 0].contiguous()), r, w, f(b)), r]
        kw = dict(D=f(b), z=f(z), dt_bias=f(b), dt_softplus=True)
        a = [f(x), f(dt), f(A), f(B), f(C)]
        out += gdr.scan_fwd(*a, initial_state=f(h0), **kw)
        out += gdr.scan_bwd(*a, f(d_y), initial_state=f(h0), d_final_state=f(h0), grad_dtype=dtype, **kw).values()
        st, one = f(h0.clone()), lambda t: f(t[:, 0].contiguous())
        kw["z"] = one(z)
        out += [gdr.scan_step(one(x), one(dt), a[2], one(B), one(C), st, **kw), st]
        out += gdr.layer_norm_fwd(f(x), f(b), f(b))
        _, mean, rstd = gdr.layer_norm_fwd(x)
        out += gdr.layer_norm_bwd(f(x), f(d_y), f(mean), f(rstd), f(b), grad_dtype=dtype).values()
        return out
    for i, (p, q) in enumerate(zip(all_of(odd), all_of(lambda t: t.clone()))):
        assert torch.isfinite(p).all() and torch.equal(p, q), i
