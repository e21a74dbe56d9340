"""More operators of a layer stack, as cases to time and to check: attention with a sliding window and a few first tokens
that stay visible (prompts, single tokens over a ring of cached rows, backward), the RMS norm of a block's heads with its
gate (forward, backward), and the residual sum with the norms before and after it (forward, backward).

With ``own`` false, ``run`` computes each in a plain form out of elementary torch operations in 32 bits; with ``own`` true
it makes the calls of the framework. ``exact`` computes the same from the definitions in 64 bits."""
import math
import random

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_DEV = "cuda:0"
_EPS = 1e-5


def listed():
    return [
        # one long prompt through a window layer
        dict(name="attn_prompt", op="attn_fwd", dtype="bf16", batch=1, tokens=65536, seqs=1, heads=32, kv=8, dk=128, dv=128, window=4096, sinks=4, cached=False),
        # pieces of several prompts that go on from their caches, packed, ragged
        dict(name="attn_pieces_packed", op="attn_fwd", dtype="bf16", batch=1, tokens=8191, seqs=13, heads=16, kv=4, dk=64, dv=64, window=512, sinks=4, cached=True),
        # odd sizes in fp32: three query heads to a key head, head sizes that fill no tile
        dict(name="attn_odd_f32", op="attn_fwd", dtype="f32", batch=3, tokens=3 * 1037, seqs=3, heads=6, kv=2, dk=72, dv=40, window=301, sinks=1, cached=False),
        # one decode step of 128 sequences
        dict(name="attn_decode", op="attn_step", dtype="bf16", seqs=128, heads=32, kv=8, dk=128, dv=128, window=4096, sinks=4),
        # one token of one sequence: latency
        dict(name="attn_decode_one", op="attn_step", dtype="bf16", seqs=1, heads=16, kv=4, dk=128, dv=128, window=1024, sinks=4),
        # a training step of a window layer, 4 sequences of 4096
        dict(name="attn_train", op="attn_bwd", dtype="bf16", batch=4, tokens=16384, seqs=4, heads=16, kv=4, dk=128, dv=128, window=1024, sinks=4),
        # training on packed documents of uneven lengths, one key head to every query head
        dict(name="attn_train_packed", op="attn_bwd", dtype="bf16", batch=1, tokens=6001, seqs=17, heads=8, kv=8, dk=64, dv=64, window=256, sinks=1),
        # the gated norm of every head's output of a long prompt (32 heads of 128)
        dict(name="gated_heads", op="gated_fwd", dtype="bf16", rows=65536 * 32, cols=128),
        # the same in a training step of 16,384 tokens
        dict(name="gated_train", op="gated_bwd", dtype="bf16", rows=16384 * 32, cols=128),
        # between two blocks of a decode batch, the residual stream in fp32
        dict(name="residual_decode", op="residual_fwd", dtype="bf16", stream="f32", rows=256, cols=4096, post=False, gate="none"),
        # a prompt through norms on both sides of a block with a gate per channel
        dict(name="residual_prompt", op="residual_fwd", dtype="bf16", stream="bf16", rows=16384, cols=4096, post=True, gate="channel"),
        # a training step at the model's width, everything on, a gate per token
        dict(name="residual_train", op="residual_bwd", dtype="bf16", stream="bf16", rows=16384, cols=4096, post=True, gate="token"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    """One more case: sizes over the ranges that the listed ones span, odd ones among them."""
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_step", "attn_bwd", "gated_fwd", "gated_bwd", "residual_fwd", "residual_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("gated"):
        cols = rng.choice([32, 64, 128, 128, 256, _log(rng, 17, 1024)])
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, (1 << 27) // cols), cols=cols)
    if op.startswith("residual"):
        cols = _log(rng, 64, 8192)
        cols = cols if rng.random() < 0.3 else max(64, cols // 64 * 64)
        return dict(op=op, dtype=dtype, stream=rng.choice([dtype, "f32"]), rows=_log(rng, 1, (1 << 26) // cols), cols=cols,
                    post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token"]))
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    dk = rng.choice([32, 64, 64, 128, 128, 128, 72, 80, 96])
    dv = dk if rng.random() < 0.8 else rng.choice([32, 64, 128])
    window, sinks = _log(rng, 1, 4096), rng.choice([0, 1, 4, 4, 16, 70])
    shape = dict(heads=heads, kv=kv, dk=dk, dv=dv, window=window, sinks=sinks)
    if op == "attn_step":
        return dict(op=op, dtype=dtype, seqs=_log(rng, 1, min(512, (1 << 28) // ((window + sinks) * kv * dk))), **shape)
    # fp32 and backward passes get a smaller share of the largest prompt's products
    most = 65536 * 4096 * 32 * 128 // (16 if dtype == "f32" else 4)
    tokens = _log(rng, 1, min(32768, max(1, most // (min(window + sinks, 4096) * heads * dk)), (1 << 27) // (heads * dk)))
    seqs = _log(rng, 1, min(32, tokens))
    batch = seqs if rng.random() < 0.5 else 1
    tokens = tokens // batch * batch
    case = dict(op=op, dtype=dtype, batch=batch, tokens=tokens, seqs=seqs, **shape)
    if op == "attn_fwd":
        case["cached"] = rng.random() < 0.5
    return case


def _offsets(case):
    """Sequence offsets: equal rows of a batch, or ragged cuts of the packed tokens (some of them empty)."""
    if case["batch"] == case["seqs"]:
        n = case["tokens"] // case["batch"]
        return [i * n for i in range(case["batch"] + 1)]
    r = random.Random(case["tokens"] * 131 + case["seqs"])
    cuts = sorted(r.randint(0, case["tokens"]) for _ in range(case["seqs"] - 1))
    return [0] + cuts + [case["tokens"]]


def _lens(case):
    """Tokens that each sequence has behind it: some none, some less than a window, some several."""
    N, W, S = case["seqs"], case["window"], case["sinks"]
    if case["op"] != "attn_step" and not case["cached"]:
        return [0] * N
    r = random.Random(N * 977 + W)
    if case["op"] == "attn_step":
        return [r.randint(W // 2, 3 * W + S) for _ in range(N)]
    return [0 if i % 5 == 4 else r.randint(0, 3 * W + S) for i in range(N)]


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    t = _T[case["dtype"]]

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device=_DEV, dtype=torch.float32).mul_(std).add_(mean).to(dtype)

    op, s = case["op"], dict(case=case)
    if op.startswith("gated"):
        R, C = case["rows"], case["cols"]
        s.update(x=normal(R, C, dtype=t, std=0.5), z=normal(R, C, dtype=t, std=1.5), weight=normal(C, std=0.2, mean=1.0))
        if op == "gated_bwd":      # what a training step keeps of the forward pass
            s["rstd"] = (s["x"].float().square().mean(1) + _EPS).rsqrt()
            s["d_y"] = normal(R, C, dtype=t)
        return s
    if op.startswith("residual"):
        R, C, stream = case["rows"], case["cols"], _T[case["stream"]]
        s.update(x=normal(R, C, dtype=t, std=0.7), weight=normal(C, std=0.2, mean=1.0), scale=0.5,
                 x_weight=normal(C, std=0.2, mean=1.0) if case["post"] else None,
                 gate=dict(none=lambda: None, channel=lambda: normal(C, std=0.3, mean=0.5),
                           token=lambda: normal(R, C, dtype=t, std=0.3, mean=0.5))[case["gate"]]())
        if op == "residual_fwd":
            s["residual"] = normal(R, C, dtype=stream, std=2.0)
        else:
            s["h"] = normal(R, C, dtype=stream, std=2.0)
            s["rstd"] = (s["h"].float().square().mean(1) + _EPS).rsqrt()
            s["x_rstd"] = (s["x"].float().square().mean(1) + _EPS).rsqrt() if case["post"] else None
            s["d_y"], s["d_h"] = normal(R, C, dtype=t), normal(R, C, dtype=stream)
        return s
    N, H, K, dk, dv = case["seqs"], case["heads"], case["kv"], case["dk"], case["dv"]
    if op == "attn_step":
        lead = (N,)
    else:
        off = _offsets(case)
        packed = case["batch"] != N
        lead = (case["batch"], case["tokens"] // case["batch"])
        s.update(off=off, cu_cpu=torch.tensor(off, dtype=torch.int32) if packed else None,
                 cu=torch.tensor(off, dtype=torch.int32, device=_DEV) if packed else None)
    s.update(q=normal(*lead, H, dk, dtype=t), k=normal(*lead, K, dk, dtype=t), v=normal(*lead, K, dv, dtype=t))
    if op != "attn_bwd":
        s["past"] = _lens(case)
        if op == "attn_step" or case["cached"]:
            rows = case["sinks"] + case["window"]
            s["cache"] = (normal(N, rows, K, dk, dtype=t), normal(N, rows, K, dv, dtype=t))
            s["lens"] = torch.tensor(s["past"], dtype=torch.int32, device=_DEV)
        else:
            s["cache"] = s["lens"] = None
    else:
        s["past"] = [0] * N
        s["o"], s["lse"] = _attn_prompt(dict(s, cache=None))     # what a training step keeps of the forward pass
        s["d_o"] = normal(*lead, H, dv, dtype=t)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _slots(positions, W, S):
    return torch.where(positions < S, positions, S + (positions - S) % W)


def _history(s, n):
    """Positions whose rows the cache of sequence n holds, ascending."""
    W, S, past = s["case"]["window"], s["case"]["sinks"], s["past"][n]
    return torch.cat([torch.arange(min(S, past), device=_DEV), torch.arange(max(S, past - W), max(S, past), device=_DEV)])


def _blocks(s):
    """For every sequence and run of its queries: (sequence, first query, one past the last, keys' positions)."""
    W, S = s["case"]["window"], s["case"]["sinks"]
    step = min(1024, max(64, W // 2))
    for n in range(len(s["off"]) - 1):
        a, b, past = s["off"][n], s["off"][n + 1], s["past"][n]
        for i in range(a, b, step):
            j = min(i + step, b)
            lo, hi = max(S, past + i - a - W + 1), past + j - a
            yield n, i, j, torch.cat([torch.arange(min(S, hi), device=_DEV), torch.arange(lo, max(lo, hi), device=_DEV)])


def _rows(s, n, what, positions):
    """The rows of k (0) or v (1) at these positions of sequence n, heads first: [kv, positions, d]."""
    x = s["k" if what == 0 else "v"]
    x = x.reshape((-1,) + x.shape[2:])
    a, past = s["off"][n], s["past"][n]
    if past == 0:
        return x[a + positions].float().transpose(0, 1).contiguous()
    old = positions < past
    row = x[(a + positions - past).clamp(min=a, max=x.shape[0] - 1)]
    kept = s["cache"][what][n][_slots(positions, s["case"]["window"], s["case"]["sinks"])]
    return torch.where(old[:, None, None], kept, row).float().transpose(0, 1).contiguous()


def _scores(s, n, i, j, pos, K):
    """Scores of queries i..j - 1 against the keys K at these positions, -inf where a key is not seen: [kv, G, queries, keys]."""
    case = s["case"]
    q = s["q"].reshape(-1, case["kv"], case["heads"] // case["kv"], case["dk"])[i:j].float().permute(1, 2, 0, 3)
    t = torch.arange(i, j, device=_DEV) - s["off"][n] + s["past"][n]
    d = t[:, None] - pos[None]
    seen = (d >= 0) & ((d < case["window"]) | (pos[None] < case["sinks"]))
    v = torch.matmul(q.reshape(case["kv"], -1, case["dk"]), K.transpose(1, 2).contiguous()) * case["dk"] ** -0.5
    return v.reshape(case["kv"], -1, j - i, pos.numel()).masked_fill_(~seen, float("-inf"))


def _attn_prompt(s):
    case, q = s["case"], s["q"]
    kv, G, dv = case["kv"], case["heads"] // case["kv"], case["dv"]
    o = torch.empty((q.shape[0] * q.shape[1], kv, G, dv), dtype=q.dtype, device=_DEV)
    lse = torch.empty(o.shape[:3], device=_DEV)
    for n, i, j, pos in _blocks(s):
        v = _scores(s, n, i, j, pos, _rows(s, n, 0, pos))
        m = v.amax(3, keepdim=True)
        e = torch.exp_(v.sub_(m))
        l = e.sum(3, keepdim=True)
        out = torch.matmul(e.reshape(kv, -1, pos.numel()), _rows(s, n, 1, pos)).reshape(kv, G, j - i, dv) / l
        o[i:j] = out.permute(2, 0, 1, 3).to(q.dtype)
        lse[i:j] = (m + torch.log(l))[..., 0].permute(2, 0, 1)
    return o.reshape(q.shape[:3] + (dv,)), lse.reshape(q.shape[:3])


def _keep(s):
    """The cache after the new tokens: those among the first ones and the last window of the rest."""
    W, S = s["case"]["window"], s["case"]["sinks"]
    for n in range(len(s["off"]) - 1):
        a, b, past = s["off"][n], s["off"][n + 1], s["past"][n]
        end = past + b - a
        first = torch.arange(past, max(past, min(S, end)), device=_DEV)
        pos = torch.cat([first, torch.arange(max(S, past, end - W), max(end, S, past), device=_DEV)])
        for c, x in zip(s["cache"], (s["k"], s["v"])):
            c[n][_slots(pos, W, S)] = x.reshape((-1,) + x.shape[2:])[a + pos - past]


def _attn_step(s):
    case, q = s["case"], s["q"]
    N, kv, G, dk, W, S = case["seqs"], case["kv"], case["heads"] // case["kv"], case["dk"], case["window"], case["sinks"]
    t = s["lens"].long()
    for c, x in zip(s["cache"], (s["k"], s["v"])):
        c[torch.arange(N, device=_DEV), _slots(t, W, S)] = x
    K, V = (c.float().transpose(1, 2).contiguous() for c in s["cache"])
    v = torch.matmul(q.float().reshape(N, kv, G, dk), K.transpose(2, 3).contiguous()) * dk ** -0.5
    held = torch.arange(S + W, device=_DEV)[None] <= t[:, None]
    v.masked_fill_(~held[:, None, None], float("-inf"))
    e = torch.exp(v - v.amax(3, keepdim=True))
    o = torch.matmul(e, V) / e.sum(3, keepdim=True)
    return [o.reshape(N, case["heads"], -1).to(q.dtype), *s["cache"]]


def _attn_grads(s):
    case, q = s["case"], s["q"]
    kv, G, dk, dv = case["kv"], case["heads"] // case["kv"], case["dk"], case["dv"]
    scale = dk ** -0.5
    n_all = q.shape[0] * q.shape[1]
    dq = torch.empty((n_all, kv, G, dk), dtype=q.dtype, device=_DEV)
    dK, dV = torch.zeros((kv, n_all, dk), device=_DEV), torch.zeros((kv, n_all, dv), device=_DEV)
    d_o, o = (s[x].reshape(-1, kv, G, dv) for x in ("d_o", "o"))
    lse = s["lse"].reshape(-1, kv, G)
    for n, i, j, pos in _blocks(s):
        K, V = _rows(s, n, 0, pos), _rows(s, n, 1, pos)
        p = torch.exp_(_scores(s, n, i, j, pos, K).sub_(lse[i:j].permute(1, 2, 0)[..., None])).reshape(kv, -1, pos.numel())
        g = d_o[i:j].float()
        delta = (g * o[i:j].float()).sum(3).permute(1, 2, 0).reshape(kv, -1, 1)
        g = g.permute(1, 2, 0, 3).reshape(kv, -1, dv)
        ds = torch.matmul(g, V.transpose(1, 2).contiguous()).sub_(delta).mul_(p).mul_(scale)
        at = pos + s["off"][n]
        dq[i:j] = torch.matmul(ds, K).reshape(kv, G, j - i, dk).permute(2, 0, 1, 3).to(q.dtype)
        qf = s["q"].reshape(-1, kv, G, dk)[i:j].float().permute(1, 2, 0, 3).reshape(kv, -1, dk)
        dK.index_add_(1, at, torch.matmul(ds.transpose(1, 2).contiguous(), qf))
        dV.index_add_(1, at, torch.matmul(p.transpose(1, 2).contiguous(), g))
    back = lambda x, like: x.transpose(0, 1).reshape(like.shape).to(q.dtype)
    return dict(dq=dq.reshape(q.shape), dk=back(dK, s["k"]), dv=back(dV, s["v"]))


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _gated_plain(s):
    x, z, w = s["x"].float(), s["z"].float(), s["weight"]
    sg = _sigmoid(z)
    if s["case"]["op"] == "gated_fwd":
        rstd = (x.square().mean(1) + _EPS).rsqrt()
        return [(x * rstd[:, None] * w * (z * sg)).to(s["x"].dtype), rstd]
    rstd, d_y = s["rstd"][:, None], s["d_y"].float()
    hat = x * rstd
    da = d_y * (z * sg)
    c = da * w
    dx = rstd * (c - hat * (c * hat).mean(1, keepdim=True))
    dz = d_y * hat * w * (sg * (1 + z * (1 - sg)))
    return dict(dx=dx.to(s["x"].dtype), dz=dz.to(s["x"].dtype), dweight=(da * hat).sum(0))


def _residual_plain(s):
    x, w, xw, scale = s["x"].float(), s["weight"], s["x_weight"], s["scale"]
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    if s["case"]["op"] == "residual_fwd":
        a, out = x, {}
        if xw is not None:
            out["x_rstd"] = (x.square().mean(1) + _EPS).rsqrt()
            a = x * out["x_rstd"][:, None] * xw
        h = s["residual"].float() + scale * (gate * a)
        rstd = (h.square().mean(1) + _EPS).rsqrt()
        out.update(y=(h * rstd[:, None] * w).to(s["x"].dtype), h=h.to(s["residual"].dtype), rstd=rstd)
        return out
    hat, d_y = s["h"].float() * s["rstd"][:, None], s["d_y"].float()
    c = d_y * w
    dh = s["d_h"].float() + s["rstd"][:, None] * (c - hat * (c * hat).mean(1, keepdim=True))
    out = dict(dresidual=dh.to(s["h"].dtype), dweight=(d_y * hat).sum(0))
    da = scale * gate * dh
    if xw is not None:
        xr = s["x_rstd"][:, None]
        xhat = x * xr
        a = xhat * xw
        out["dx_weight"] = (da * xhat).sum(0)
        c = da * xw
        dx = xr * (c - xhat * (c * xhat).mean(1, keepdim=True))
    else:
        a, dx = x, da
    out["dx"] = dx.to(s["x"].dtype)
    if s["gate"] is not None:
        dg = scale * a * dh
        out["dgate"] = dg.sum(0) if s["gate"].dim() == 1 else dg.to(s["x"].dtype)
    return out


# ------------------------------------------------------------------------------------------------ the framework's calls
def _call(s):
    import chunkwise_gated_delta_local_amd as gdr
    case, op = s["case"], s["case"]["op"]
    if op == "gated_fwd":
        return list(gdr.gated_norm_fwd(s["x"], s["z"], s["weight"]))
    if op == "gated_bwd":
        return gdr.gated_norm_bwd(s["x"], s["z"], s["d_y"], s["rstd"], s["weight"], grad_dtype=s["x"].dtype)
    if op == "residual_fwd":
        y, h, rstd, x_rstd = gdr.residual_norm_fwd(s["x"], s["residual"], s["weight"], x_weight=s["x_weight"],
                                                   gate=s["gate"], scale=s["scale"])
        out = dict(y=y, h=h, rstd=rstd)
        if x_rstd is not None:
            out["x_rstd"] = x_rstd
        return out
    if op == "residual_bwd":
        return gdr.residual_norm_bwd(s["x"], s["h"], s["d_y"], s["rstd"], s["weight"], d_h=s["d_h"], x_weight=s["x_weight"],
                                     x_rstd=s["x_rstd"], gate=s["gate"], scale=s["scale"], grad_dtype=s["x"].dtype)
    W, S = case["window"], case["sinks"]
    if op == "attn_step":
        return [gdr.window_attn_step(s["q"], s["k"], s["v"], s["cache"], s["lens"], W, S), *s["cache"]]
    seqs = dict(cu_seqlens=s["cu"], cu_seqlens_cpu=s["cu_cpu"])
    if op == "attn_bwd":
        return gdr.window_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["d_o"], W, S, grad_dtype=s["q"].dtype, **seqs)
    return [*gdr.window_attn_fwd(s["q"], s["k"], s["v"], W, S, cache=s["cache"], lens=s["lens"], **seqs), *(s["cache"] or ())]


def run(state):
    if own:
        return _call(state)
    op = state["case"]["op"]
    if op.startswith("gated"):
        return _gated_plain(state)
    if op.startswith("residual"):
        return _residual_plain(state)
    if op == "attn_step":
        return _attn_step(state)
    if op == "attn_bwd":
        return _attn_grads(state)
    out = list(_attn_prompt(state))
    if state["cache"] is None:
        return out
    _keep(state)
    return out + list(state["cache"])


# ------------------------------------------------------------------------------------------------ work
def _sum_min(a, b, most):
    """sum over p in [a, b) of min(p + 1, most)"""
    m = min(max(most, a), b)                    # p + 1 <= most for p < most
    return (m * (m + 1) - a * (a + 1)) // 2 + (b - m) * most


def _pairs(case, off, past):
    """(query, key) pairs that are seen, and rows of the caches that some query sees."""
    W, S = case["window"], case["sinks"]
    pairs = rows = 0
    for n in range(len(off) - 1):
        a, b = past[n], past[n] + off[n + 1] - off[n]
        # a query at p sees min(p + 1, W + S) keys
        pairs += _sum_min(a, b, W + S)
        rows += min(a, S + W - 1) if b > a else 0
    return pairs, rows


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("gated"):
        R, C = case["rows"], case["cols"]
        if op == "gated_fwd":
            return {"bytes": 3 * e * R * C + 4 * C + 4 * R, "flops": 10 * R * C}
        return {"bytes": 5 * e * R * C + 8 * C + 4 * R, "flops": 22 * R * C}
    if op.startswith("residual"):
        R, C, r = case["rows"], case["cols"], 2 if case["stream"] == "bf16" else 4
        norms, token = 1 + int(case["post"]), int(case["gate"] == "token")
        if op == "residual_fwd":
            return {"bytes": R * C * (2 * e + 2 * r + token * e) + 4 * C * (norms + 1) + 4 * R * norms, "flops": R * C * (3 + 4 * norms)}
        return {"bytes": R * C * (3 * e + 3 * r + 2 * token * e) + 8 * C * (norms + 1) + 4 * R * norms, "flops": R * C * (4 + 9 * norms)}
    H, K, dk, dv, N = case["heads"], case["kv"], case["dk"], case["dv"], case["seqs"]
    if op == "attn_step":
        past = _lens(case)
        seen = sum(min(p + 1, case["window"] + case["sinks"]) for p in past)
        return {"bytes": e * (seen * K * (dk + dv) + N * (H + K) * (dk + dv)) + 4 * N, "flops": 2 * seen * H * (dk + dv)}
    off, n = _offsets(case), case["tokens"]
    if op == "attn_bwd":
        pairs, _ = _pairs(case, off, [0] * N)
        return {"bytes": e * n * (2 * H * (dk + dv) + 2 * K * (dk + dv)) + 4 * n * H, "flops": pairs * H * (6 * dk + 4 * dv)}
    pairs, rows = _pairs(case, off, _lens(case))
    moved = n * (H + K) * (dk + dv)
    if case["cached"]:
        kept = sum(min(off[i + 1] - off[i], case["window"] + case["sinks"]) for i in range(N))
        moved += (rows + kept) * K * (dk + dv)
    return {"bytes": e * moved + 4 * n * H, "flops": 2 * pairs * H * (dk + dv)}


# ------------------------------------------------------------------------------------------------ 64 bits
def _exact_rms(x):
    return 1 / torch.sqrt((x * x).sum(-1) / x.shape[-1] + _EPS)


def _exact_rms_grad(g, hat, r):
    return r[:, None] * (g - hat * ((g * hat).sum(1) / g.shape[1])[:, None])


def _exact_gated(s):
    x, z, w = s["x"].double(), s["z"].double(), s["weight"].double()
    sg = torch.sigmoid(z)
    if s["case"]["op"] == "gated_fwd":
        r = _exact_rms(x)
        return [x.mul_(r[:, None]).mul_(w).mul_(z.mul_(sg)), r]
    r, dy = s["rstd"].double(), s["d_y"].double()
    hat = x * r[:, None]
    dn = dy * z * sg
    return dict(dx=_exact_rms_grad(dn * w, hat, r), dz=dy * hat * w * (sg + z * sg * (1 - sg)), dweight=(dn * hat).sum(0))


def _exact_residual(s):
    x, w, f = s["x"].double(), s["weight"].double(), s["scale"]
    if s["gate"] is not None:
        f = f * s["gate"].double()
    xw = None if s["x_weight"] is None else s["x_weight"].double()
    if s["case"]["op"] == "residual_fwd":
        out, a = {}, x
        if xw is not None:
            out["x_rstd"] = _exact_rms(x)
            a = x * out["x_rstd"][:, None] * xw
        h = s["residual"].double() + f * a
        r = _exact_rms(h)
        out.update(y=h * r[:, None] * w, h=h, rstd=r)
        return out
    r, dy = s["rstd"].double(), s["d_y"].double()
    hat = s["h"].double() * r[:, None]
    dh = s["d_h"].double() + _exact_rms_grad(dy * w, hat, r)
    out = dict(dresidual=dh, dweight=(dy * hat).sum(0))
    a, db = x, f * dh
    out["dx"] = db
    if xw is not None:
        xr = s["x_rstd"].double()
        xhat = x * xr[:, None]
        a = xhat * xw
        out["dx_weight"] = (db * xhat).sum(0)
        out["dx"] = _exact_rms_grad(db * xw, xhat, xr)
    if s["gate"] is not None:
        dg = s["scale"] * dh * a
        out["dgate"] = dg if s["gate"].dim() == 2 else dg.sum(0)
    return out


def _exact_attn(s):
    """Query by query of the definition, some of them side by side: each reads the rows lo..hi of its sequence's tokens (the
    cached ones laid out in order before the new ones) and masks what it does not see."""
    case, op = s["case"], s["case"]["op"]
    H, kv, dk, W, S = case["heads"], case["kv"], case["dk"], case["window"], case["sinks"]
    G, scale = H // kv, dk ** -0.5
    off = s["off"] if "off" in s else list(range(case["seqs"] + 1))
    flat = {x: s[x].reshape((-1,) + s[x].shape[-2:]) for x in ("q", "k", "v")}
    n_all = flat["q"].shape[0]
    o = torch.empty(n_all, H, case["dv"], dtype=torch.float64, device=_DEV)
    lse = torch.empty(n_all, H, dtype=torch.float64, device=_DEV)
    grads = None
    if op == "attn_bwd":
        grads = dict(dq=torch.zeros(flat["q"].shape, dtype=torch.float64, device=_DEV),
                     dk=torch.zeros(flat["k"].shape, dtype=torch.float64, device=_DEV),
                     dv=torch.zeros(flat["v"].shape, dtype=torch.float64, device=_DEV))
    after = None if s.get("cache") is None else [c.double() for c in s["cache"]]
    for n in range(len(off) - 1):
        a, b, past = off[n], off[n + 1], s["past"][n]
        if a == b:
            continue
        # old[i] is the position of row i before the new tokens
        old = [p for p in range(past) if p < S or p >= past - W] if past else []
        where = [p if p < S else S + (p - S) % W for p in old]
        pos = torch.tensor(old + list(range(past, past + b - a)), device=_DEV)
        rows = []
        for i, x in enumerate(("k", "v")):
            new = flat[x][a:b].double()
            rows.append(torch.cat([after[i][n][torch.tensor(where, dtype=torch.long, device=_DEV)], new]) if old else new)
        step = max(1, min(512, (1 << 27) // (H * min(pos.numel(), W + S + 512))))
        for i in range(a, b, step):
            j = min(i + step, b)
            p = torch.arange(i - a + past, j - a + past, device=_DEV)
            near = (pos < S) | ((pos <= int(p[-1])) & (pos > int(p[0]) - W))
            at = near.nonzero()[:, 0]
            behind = p[:, None] - pos[at][None]
            hide = (behind < 0) | ((behind >= W) & (pos[at][None] >= S))
            for g in range(kv):
                heads = slice(g * G, (g + 1) * G)
                q = flat["q"][i:j, heads].double()                        # [queries, G, dk]
                K, V = rows[0][at, g], rows[1][at, g]
                sc = (q.reshape(-1, dk) @ K.t()).reshape(j - i, G, -1) * scale
                sc[hide[:, None].expand_as(sc)] = -math.inf
                if grads is None:
                    top = torch.logsumexp(sc, 2)
                    lse[i:j, heads] = top
                    o[i:j, heads] = (torch.exp(sc - top[..., None]).reshape(-1, at.numel()) @ V).reshape(j - i, G, -1)
                    continue
                P = torch.exp(sc - s["lse"].reshape(-1, H)[i:j, heads].double()[..., None]).reshape(-1, at.numel())
                dO = s["d_o"].reshape(-1, H, case["dv"])[i:j, heads].double().reshape(-1, case["dv"])
                O = s["o"].reshape(-1, H, case["dv"])[i:j, heads].double().reshape(-1, case["dv"])
                dS = P * (dO @ V.t() - (dO * O).sum(1, keepdim=True)) * scale
                grads["dq"][i:j, heads] = (dS @ K).reshape(j - i, G, dk)
                grads["dk"][a + at, g] += dS.t() @ q.reshape(-1, dk)
                grads["dv"][a + at, g] += P.t() @ dO
        if after is not None:
            last = {t if t < S else S + (t - S) % W: t - past for t in range(past, past + b - a)}     # slot: its last token
            slot, tok = (torch.tensor(list(x), device=_DEV) for x in (last.keys(), last.values()))
            for c, x in zip(after, ("k", "v")):
                c[n][slot] = flat[x][a + tok].double()
    if grads is not None:
        return {x: grads[x].reshape(s[x[1:]].shape) for x in ("dq", "dk", "dv")}
    o = o.reshape(s["q"].shape[:-1] + (case["dv"],))
    return [o, *after] if op == "attn_step" else [o, lse.reshape(s["q"].shape[:-1]), *(after or ())]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_gated(s) if op.startswith("gated") else _exact_residual(s) if op.startswith("residual") else _exact_attn(s)
