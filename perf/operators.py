"""The layer operators around the gated delta rule, as cases to time and to check: the short causal convolution, the
selective state space scan (each for prompts, for single tokens and backward) and layer norm (forward and backward).

With ``own`` false, ``run`` computes each in a plain form out of elementary torch operations in 32 bits; with ``own`` true
it makes the calls of the framework. ``exact`` computes the same from the definitions in 64 bits."""
import math
import random

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_DEV = "cuda:0"


def listed():
    return [
        # the projections q, k, v of a long packed prompt (16 + 16 + 32 heads of 128) before the recurrence
        dict(name="conv_prompt_packed", op="conv_fwd", dtype="bf16", batch=1, tokens=65536, seqs=9, channels=8192, width=4),
        # one decode step of 256 sequences
        dict(name="conv_decode", op="conv_step", dtype="bf16", seqs=256, channels=8192, width=4),
        # the same projections in a training step, 4 sequences of 4096 with 16 heads of 128 each
        dict(name="conv_train", op="conv_bwd", dtype="bf16", batch=4, tokens=16384, seqs=4, channels=6144, width=4),
        # one prompt through the scan, with the output gate
        dict(name="scan_prompt", op="scan_fwd", dtype="bf16", batch=1, tokens=8192, seqs=1, channels=4096, state=16, groups=1, gate=True),
        # ragged packed prompts in fp32 with odd sizes and grouped B and C
        dict(name="scan_packed_f32", op="scan_fwd", dtype="f32", batch=1, tokens=4099, seqs=13, channels=1540, state=24, groups=4, gate=False),
        # a training step of the scan
        dict(name="scan_train", op="scan_bwd", dtype="bf16", batch=4, tokens=8192, seqs=4, channels=2048, state=16, groups=1, gate=True),
        # one decode step of 256 sequences: the states read and written
        dict(name="scan_decode", op="scan_step", dtype="bf16", seqs=256, channels=4096, state=16, groups=1, gate=True),
        # one token of one sequence: latency
        dict(name="scan_decode_one", op="scan_step", dtype="bf16", seqs=1, channels=2048, state=16, groups=1, gate=True),
        # the norm of every head's output of a long prompt (32 heads of 128)
        dict(name="norm_heads", op="norm_fwd", dtype="bf16", rows=65536 * 32, cols=128),
        # a decode batch at the model's width
        dict(name="norm_decode", op="norm_fwd", dtype="bf16", rows=256, cols=4096),
        # training at the model's width
        dict(name="norm_train", op="norm_bwd", dtype="bf16", rows=16384, cols=4096),
        # odd sizes in fp32
        dict(name="norm_odd_f32", op="norm_bwd", dtype="f32", rows=4001, cols=2561),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the ranges that the listed ones span, odd ones among them."""
    op = rng.choice(["conv_fwd", "conv_step", "conv_bwd", "scan_fwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        cols = _log(rng, 32, 8192)
        cols = cols if rng.random() < 0.3 else max(32, cols // 32 * 32)
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, min(1 << 21, (1 << 26) // cols)), cols=cols)
    width = rng.choice([2, 3, 4, 4])
    channels = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        channels = max(64, channels // 64 * 64)
    if op == "conv_step":
        return dict(op=op, dtype=dtype, seqs=_log(rng, 1, 512), channels=channels, width=width)
    if op.startswith("conv"):
        tokens = _log(rng, 1, min(65536, (1 << 27) // channels))
        seqs = _log(rng, 1, min(64, tokens))
        batch = seqs if rng.random() < 0.5 else 1
        tokens = tokens // batch * batch
        return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, seqs=seqs, channels=channels, width=width)
    state = rng.choice([8, 16, 16, 16, 20, 32, 64])
    groups = rng.choice([1, 1, 2, 4])
    channels = max(groups, min(channels, 4096) // groups * groups)
    gate = rng.random() < 0.7
    if op == "scan_step":
        return dict(op=op, dtype=dtype, seqs=_log(rng, 1, 512), channels=channels, state=state, groups=groups, gate=gate)
    tokens = _log(rng, 1, min(16384, (1 << 27) // (channels * state)))
    seqs = _log(rng, 1, min(32, tokens))
    batch = seqs if rng.random() < 0.5 else 1
    tokens = tokens // batch * batch
    return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, seqs=seqs, channels=channels, state=state, groups=groups, gate=gate)


def _offsets(case):
    """Sequence offsets: equal rows of a batch, or ragged cuts of the packed tokens (some of them empty)."""
    if case["batch"] == case["seqs"]:
        n = case["tokens"] // case["batch"]
        return [i * n for i in range(case["batch"] + 1)]
    r = random.Random(case["tokens"] * 131 + case["seqs"])
    cuts = sorted(r.randint(0, case["tokens"]) for _ in range(case["seqs"] - 1))
    return [0] + cuts + [case["tokens"]]


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    t = _T[case["dtype"]]

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device=_DEV, dtype=torch.float32).mul_(std).add_(mean).to(dtype)

    op, s = case["op"], dict(case=case)
    if op.startswith("norm"):
        R, C = case["rows"], case["cols"]
        s.update(x=normal(R, C, dtype=t, std=1.5, mean=0.3), weight=normal(C, std=0.2, mean=1.0), bias=normal(C, std=0.2))
        if op == "norm_bwd":      # what a training step keeps of the forward pass
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = (x - s["mean"][:, None]).square().mean(1).add(1e-5).rsqrt()
            s["d_y"] = normal(R, C, dtype=t)
        return s
    D, N = case["channels"], case["seqs"]
    if "batch" in case:
        off = _offsets(case)
        B, T = case["batch"], case["tokens"] // case["batch"]
        packed = B != N
        s.update(off=off, lead=(B, T), cu_cpu=torch.tensor(off, dtype=torch.int32) if packed else None,
                 cu=torch.tensor(off, dtype=torch.int32, device=_DEV) if packed else None)
        s["starts"] = torch.tensor(off[:-1], device=_DEV)
        s["ends"] = torch.tensor(off[1:], device=_DEV)
        s["seq"] = torch.repeat_interleave(torch.arange(N, device=_DEV), s["ends"] - s["starts"])
        lead = (B, T)
    else:
        lead = (N,)
    if op.startswith("conv"):
        W = case["width"]
        s.update(x=normal(*lead, D, dtype=t), weight=normal(D, W, std=W ** -0.5), bias=normal(D, std=0.1),
                 state=normal(N, W - 1, D, dtype=t))
        if op == "conv_bwd":
            s.update(d_y=normal(*lead, D, dtype=t), d_final=normal(N, W - 1, D, dtype=t))
        return s
    S, G = case["state"], case["groups"]
    s.update(x=normal(*lead, D, dtype=t), dt=normal(*lead, D, dtype=t, std=0.5),
             A=-torch.exp(torch.log(torch.arange(1, S + 1, device=_DEV).float())[None] + normal(D, S, std=0.1)),
             B=normal(*lead, G, S, dtype=t), C=normal(*lead, G, S, dtype=t), D=normal(D, std=0.2, mean=1.0),
             z=normal(*lead, D, dtype=t) if case["gate"] else None,
             # softplus of the bias lies between 0.001 and 0.1
             dt_bias=torch.log(torch.expm1(torch.exp(torch.rand(D, generator=gen, device=_DEV) * math.log(100.0) + math.log(0.001)))),
             state=normal(N, D, S, std=0.5))
    if op == "scan_bwd":
        s.update(d_y=normal(*lead, D, dtype=t), d_final=normal(N, D, S, std=0.5))
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _silu(v):
    return v / (1 + torch.exp(-v))


def _dsilu(v):
    g = 1 / (1 + torch.exp(-v))
    return g * (1 + v * (1 - g))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _conv_sources(s):
    """For each tap w: the row of (tokens | initial rows) that token t reads."""
    W, n = s["case"]["width"], s["seq"].numel()
    t = torch.arange(n, device=_DEV)
    start = s["starts"][s["seq"]]
    src = t[None] - (W - 1) + torch.arange(W, device=_DEV)[:, None]
    return torch.where(src >= start, src, n + s["seq"] * (W - 1) + (src - start + W - 1))


def _conv_final_sources(s):
    W, n = s["case"]["width"], s["seq"].numel()
    src = s["ends"][:, None] - (W - 1) + torch.arange(W - 1, device=_DEV)
    q = torch.arange(s["ends"].numel(), device=_DEV)[:, None]
    return torch.where(src >= s["starts"][:, None], src, n + q * (W - 1) + (src - s["starts"][:, None] + W - 1))


def _conv_plain(s):
    case, w, b = s["case"], s["weight"], s["bias"]
    D, W, op = case["channels"], case["width"], case["op"]
    if op == "conv_step":
        u = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
        p = (u * w.t()).sum(1) + b
        y = _silu(p).to(s["x"].dtype)
        s["state"].copy_(u[:, 1:])
        return [y, s["state"]]
    rows = torch.cat([s["x"].reshape(-1, D), s["state"].reshape(-1, D)])
    n, src = s["seq"].numel(), _conv_sources(s)
    p = sum(rows[src[i]].float() * w[:, i] for i in range(W)) + b
    if op == "conv_fwd":
        return [_silu(p).to(s["x"].dtype).reshape(s["x"].shape), rows[_conv_final_sources(s)]]
    dp = _dsilu(p).mul_(s["d_y"].reshape(-1, D).float())
    d_rows = torch.zeros(rows.shape, device=_DEV)
    d_rows.index_add_(0, _conv_final_sources(s).reshape(-1), s["d_final"].reshape(-1, D).float())
    dw = []
    for i in range(W):           # each row is read once by a tap
        d_rows[src[i]] += dp * w[:, i]
        dw.append((dp * rows[src[i]].float()).sum(0))
    return dict(dx=d_rows[:n].to(s["x"].dtype).reshape(s["x"].shape), dweight=torch.stack(dw, 1), dbias=dp.sum(0),
                dh0=d_rows[n:].to(s["x"].dtype).reshape(s["state"].shape))


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling (overwrites both)."""
    k, n = 1, a.shape[0]
    while k < n:
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _scan_terms(s):
    case = s["case"]
    D, S, G = case["channels"], case["state"], case["groups"]
    x = s["x"].reshape(-1, D).float()
    pre = s["dt"].reshape(-1, D).float() + s["dt_bias"]
    delta = _softplus(pre)
    Bf = s["B"].reshape(-1, G, 1, S).float().expand(-1, G, D // G, S).reshape(-1, D, S)
    Cf = s["C"].reshape(-1, G, 1, S).float().expand(-1, G, D // G, S).reshape(-1, D, S)
    z = None if s["z"] is None else s["z"].reshape(-1, D).float()
    return x, pre, delta, Bf, Cf, z


def _scan_plain(s):
    case, dtype = s["case"], s["x"].dtype
    D, S, G, op = case["channels"], case["state"], case["groups"], case["op"]
    x, pre, delta, Bf, Cf, z = _scan_terms(s)
    a = torch.exp(delta[:, :, None] * s["A"])
    b = (delta * x)[:, :, None] * Bf
    if op == "scan_step":
        h = a * s["state"] + b
        v = (h * Cf).sum(2) + s["D"] * x
        v = v if z is None else v * _silu(z)
        s["state"].copy_(h)
        return [v.to(dtype), s["state"]]
    n = x.shape[0]
    some = s["ends"] > s["starts"]                       # sequences with a token
    first, last = s["starts"][some], s["ends"][some] - 1
    h = b
    h[first] += a[first] * s["state"][some]
    a_in = a.clone()
    a_in[first] = 0
    h = _linear_scan(a_in, h)
    final = s["state"].clone()
    final[some] = h[last]
    v = (h * Cf).sum(2) + s["D"] * x
    if op == "scan_fwd":
        v = v if z is None else v * _silu(z)
        return [v.to(dtype).reshape(s["x"].shape), final]
    d_y = s["d_y"].reshape(-1, D).float()
    ds = d_y if z is None else d_y * _silu(z)
    g = ds[:, :, None] * Cf
    g[last] += s["d_final"][some]
    a_next = torch.zeros_like(a)
    a_next[:-1] = a[1:]
    a_next[last] = 0
    g = _linear_scan(a_next.flip(0), g.flip(0)).flip(0)
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    prev[first] = s["state"][some]
    p = a * prev
    gp = g * p
    gB = (g * Bf).sum(2)
    d_delta = x * gB + (gp * s["A"]).sum(2)
    d_dt = d_delta / (1 + torch.exp(-pre))
    dh0 = s["d_final"].clone()
    dh0[some] = a[first] * g[first]
    out = dict(dx=delta * gB + s["D"] * ds, ddt=d_dt,
               dB=((delta * x)[:, :, None] * g).reshape(n, G, D // G, S).sum(2),
               dC=(ds[:, :, None] * h).reshape(n, G, D // G, S).sum(2))
    if z is not None:
        out["dz"] = d_y * v * _dsilu(z)
    shape = dict(dx=s["x"].shape, ddt=s["x"].shape, dz=s["x"].shape, dB=s["B"].shape, dC=s["C"].shape)
    out = {k: t.to(dtype).reshape(shape[k]) for k, t in out.items()}
    out.update(dA=(gp * delta[:, :, None]).sum(0), dD=(ds * x).sum(0), ddt_bias=d_dt.sum(0), dh0=dh0)
    return out


def _norm_plain(s):
    x, w = s["x"].float(), s["weight"]
    if s["case"]["op"] == "norm_fwd":
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = (c.square().mean(1) + 1e-5).rsqrt()
        return [(c * rstd[:, None] * w + s["bias"]).to(s["x"].dtype), mean, rstd]
    d_y, rstd = s["d_y"].float(), s["rstd"][:, None]
    hat = (x - s["mean"][:, None]) * rstd
    c = d_y * w
    dx = rstd * (c - c.mean(1, keepdim=True) - hat * (c * hat).mean(1, keepdim=True))
    return dict(dx=dx.to(s["x"].dtype), dweight=(d_y * hat).sum(0), dbias=d_y.sum(0))


# ------------------------------------------------------------------------------------------------ the framework's calls
def _call(s):
    import chunkwise_gated_delta_local_amd as gdr
    op, dtype = s["case"]["op"], s["x"].dtype
    if op == "norm_fwd":
        return list(gdr.layer_norm_fwd(s["x"], s["weight"], s["bias"]))
    if op == "norm_bwd":
        return gdr.layer_norm_bwd(s["x"], s["d_y"], s["mean"], s["rstd"], s["weight"], grad_dtype=dtype)
    if op == "conv_step":
        return [gdr.conv_step(s["x"], s["state"], s["weight"], s["bias"]), s["state"]]
    if op == "conv_fwd":
        return list(gdr.conv_fwd(s["x"], s["weight"], s["bias"], initial_state=s["state"], cu_seqlens=s["cu"],
                                 cu_seqlens_cpu=s["cu_cpu"]))
    if op == "conv_bwd":
        return gdr.conv_bwd(s["x"], s["weight"], s["d_y"], s["bias"], initial_state=s["state"], d_final_state=s["d_final"],
                            cu_seqlens=s["cu"], cu_seqlens_cpu=s["cu_cpu"], grad_dtype=dtype)
    more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True)
    if op == "scan_step":
        return [gdr.scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], **more), s["state"]]
    more.update(initial_state=s["state"], cu_seqlens=s["cu"], cu_seqlens_cpu=s["cu_cpu"])
    if op == "scan_fwd":
        return list(gdr.scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], **more))
    return gdr.scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["d_y"], d_final_state=s["d_final"], grad_dtype=dtype, **more)


def run(state):
    if own:
        return _call(state)
    op = state["case"]["op"]
    return _norm_plain(state) if op.startswith("norm") else _conv_plain(state) if op.startswith("conv") else _scan_plain(state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        R, C = case["rows"], case["cols"]
        if op == "norm_fwd":
            return {"bytes": 2 * e * R * C + 8 * C + 8 * R, "flops": 8 * R * C}
        return {"bytes": 3 * e * R * C + 12 * C + 8 * R, "flops": 14 * R * C}
    D, N = case["channels"], case["seqs"]
    n = case.get("tokens", N)
    if op.startswith("conv"):
        W = case["width"]
        st = (W - 1) * D * N * e
        if op == "conv_bwd":
            return {"bytes": 3 * n * D * e + 3 * st + 8 * D * (W + 1), "flops": n * D * (6 * W + 10)}
        return {"bytes": 2 * n * D * e + 2 * st + 4 * D * (W + 1), "flops": n * D * (2 * W + 5)}
    S, G = case["state"], case["groups"]
    rows = 3 + int(case["gate"])                         # x, dt, y and z
    if op == "scan_bwd":
        rows = 5 + 2 * int(case["gate"])                 # x, dt, d_y, dx, ddt and z, dz
        return {"bytes": n * D * e * rows + 4 * n * G * S * e + 4 * D * (2 * S + 4) + 12 * N * D * S, "flops": n * D * S * 22}
    return {"bytes": n * D * e * rows + 2 * n * G * S * e + 4 * D * (S + 2) + 8 * N * D * S, "flops": n * D * S * 7}


# ------------------------------------------------------------------------------------------------ 64 bits
def _d(v):
    return None if v is None else v.double()


def _exact_norm(s):
    x = s["x"].double()
    if s["case"]["op"] == "norm_fwd":
        m = x.sum(1) / x.shape[1]
        var = ((x - m[:, None]) ** 2).sum(1) / x.shape[1]
        r = 1 / torch.sqrt(var + 1e-5)
        return [((x - m[:, None]) * r[:, None]).mul_(s["weight"].double()).add_(s["bias"].double()), m, r]
    m, r = s["mean"].double()[:, None], s["rstd"].double()[:, None]
    hat = (x - m) * r
    dy = s["d_y"].double()
    dhat = dy * s["weight"].double()
    n = x.shape[1]
    dx = r * (dhat - dhat.sum(1, True) / n - hat * ((dhat * hat).sum(1, True) / n))
    return dict(dx=dx, dweight=(dy * hat).sum(0), dbias=dy.sum(0))


def _exact_conv(s):
    case = s["case"]
    D, W, op = case["channels"], case["width"], case["op"]
    w, b, h0 = s["weight"].double(), s["bias"].double(), s["state"].double()
    if op == "conv_step":
        off, x = list(range(case["seqs"] + 1)), s["x"]
    else:
        off, x = s["off"], s["x"].reshape(-1, D)
    y, fin, dx, dh0 = [], [], [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    for q in range(len(off) - 1):
        u = torch.cat([h0[q], x[off[q]:off[q + 1]].double()])
        win = u.unfold(0, W, 1) if u.shape[0] >= W else u.new_zeros((0, D, W))       # [len, D, W]
        p = torch.einsum("tdw,dw->td", win, w) + b if win.shape[0] else u.new_zeros((0, D))
        fin.append(u[u.shape[0] - (W - 1):])
        if op != "conv_bwd":
            y.append(p * torch.sigmoid(p))
            continue
        sg = torch.sigmoid(p)
        dp = s["d_y"].reshape(-1, D)[off[q]:off[q + 1]].double() * (sg + p * sg * (1 - sg))
        dw += torch.einsum("td,tdw->dw", dp, win)
        db += dp.sum(0)
        du = torch.zeros_like(u)
        du[u.shape[0] - (W - 1):] += s["d_final"][q].double()
        for j in range(W):
            du[j:j + dp.shape[0]] += dp * w[:, j]
        dh0.append(du[:W - 1])
        dx.append(du[W - 1:])
    if op == "conv_bwd":
        return dict(dx=torch.cat(dx).reshape(s["x"].shape), dweight=dw, dbias=db, dh0=torch.stack(dh0))
    return [torch.cat(y).reshape(s["x"].shape), torch.stack(fin)]


def _exact_scan(s):
    """Token by token, the sequences side by side; a sequence that has ended keeps its state."""
    case = s["case"]
    D, S, G, N, op = case["channels"], case["state"], case["groups"], case["seqs"], case["op"]
    off = s["off"] if "off" in s else list(range(N + 1))
    longest = max(off[q + 1] - off[q] for q in range(N))
    first = torch.tensor(off[:-1], device=_DEV)
    length = torch.tensor(off[1:], device=_DEV) - first
    A, skip, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()
    flat = {k: None if s.get(k) is None else s[k].reshape((-1,) + s[k].shape[len(s["x"].shape) - 1:]) for k in ("x", "dt", "z", "B", "C", "d_y")}
    heads = lambda v: v.double().repeat_interleave(D // G, 1)                        # [N, G, S] -> [N, D, S]
    n = flat["x"].shape[0]

    def at(i):
        live = (length > i)
        row = torch.where(live, first + i, torch.zeros_like(first)).clamp(max=n - 1)
        pre = flat["dt"][row].double() + bias
        return live, row, flat["x"][row].double(), pre, torch.nn.functional.softplus(pre, threshold=1e6)

    h = s["state"].double()
    v = torch.zeros(n, D, dtype=torch.float64, device=_DEV)
    kept = []
    for i in range(longest):
        live, row, x, pre, delta = at(i)
        if op == "scan_bwd":
            kept.append(h)
        new = torch.exp(delta[:, :, None] * A) * h + (delta * x)[:, :, None] * heads(flat["B"][row])
        h = torch.where(live[:, None, None], new, h)
        v[row[live]] = ((heads(flat["C"][row]) * h).sum(2) + skip * x)[live]
    z = _d(flat["z"])
    gate = 1.0 if z is None else z * torch.sigmoid(z)
    if op != "scan_bwd":
        return [(v * gate).reshape(s["x"].shape), h]
    dy = flat["d_y"].double()
    ds_all = dy * gate
    out = {k: torch.zeros(n, D, dtype=torch.float64, device=_DEV) for k in ("dx", "ddt")}
    out.update({k: torch.zeros(n, G, S, dtype=torch.float64, device=_DEV) for k in ("dB", "dC")})
    if z is not None:
        sg = torch.sigmoid(z)
        out["dz"] = (dy * v * (sg + z * sg * (1 - sg))).reshape(s["x"].shape)
    dA, g = torch.zeros_like(A), s["d_final"].double()
    for i in reversed(range(longest)):
        live, row, x, pre, delta = at(i)
        prev, Bh, Ch = kept.pop(), heads(flat["B"][row]), heads(flat["C"][row])
        a = torch.exp(delta[:, :, None] * A)
        m = live[:, None, None].double()
        ds = ds_all[row] * m[:, :, 0]
        g = g + ds[:, :, None] * Ch
        gm = g * m
        h_t = a * prev + (delta * x)[:, :, None] * Bh
        out["dC"][row[live]] = (ds[:, :, None] * h_t).reshape(N, G, D // G, S).sum(2)[live]
        out["dB"][row[live]] = (gm * (delta * x)[:, :, None]).reshape(N, G, D // G, S).sum(2)[live]
        da = gm * prev * a                               # the gradient of delta A
        dA += (da * delta[:, :, None]).sum(0)
        gB = (gm * Bh).sum(2)
        out["dx"][row[live]] = (delta * gB + skip * ds)[live]
        out["ddt"][row[live]] = ((x * gB + (da * A).sum(2)) * torch.sigmoid(pre))[live]
        g = torch.where(live[:, None, None], a * g, g)
    out.update(dA=dA, dD=(ds_all * flat["x"].double()).sum(0), ddt_bias=out["ddt"].sum(0), dh0=g)
    for k, like in (("dx", "x"), ("ddt", "x"), ("dB", "B"), ("dC", "C")):
        out[k] = out[k].reshape(s[like].shape)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_norm(s) if op.startswith("norm") else _exact_conv(s) if op.startswith("conv") else _exact_scan(s)
