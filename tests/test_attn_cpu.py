"""The window attention without a device: what its entry points refuse before any device work, the sizes of its launches,
and its bookkeeping (which keys a block sees, which number a block has), compiled from its source for the host."""
import ctypes
import json
import os
import random
import re
import subprocess
import sys

import pytest
import torch

import chunkwise_gated_delta_local_amd as gdr
from chunkwise_gated_delta_local_amd import api
from test_launch_sizes_cpu import STAND_IN

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "chunkwise_gated_delta_local_amd", "csrc")
FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)
BIG = ctypes.c_size_t(1 << 62)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="passes placeholder addresses")


@pytest.fixture(scope="module")
def lib():
    return api.load_library()


def attn(**kw):
    d = dict(batch=2, seq_len=10, num_seqs=2, num_q_heads=4, num_kv_heads=2, head_dim_qk=64, head_dim_v=32, window=8, sinks=2,
             scale=0.125, io_dtype=1, out_dtype=1, do_dtype=1, grad_dtype=0)
    d.update(kw)
    d.setdefault("q_stride", d["num_q_heads"] * d["head_dim_qk"])
    d.setdefault("k_stride", d["num_kv_heads"] * d["head_dim_qk"])
    d.setdefault("v_stride", d["num_kv_heads"] * d["head_dim_v"])
    return api.AttnProblem(**d)


def size(lib, op, p):
    n = ctypes.c_size_t(0)
    return getattr(lib, "gdr_window_attn_%s_workspace_size" % op)(ctypes.byref(p), ctypes.byref(n)), n.value


def calls(lib, **kw):
    """name -> (function, arguments, index of every tensor argument, indices of the required ones)"""
    p, F = ctypes.byref(attn(**kw)), FAKE
    one = ctypes.byref(attn(**{**kw, "seq_len": 1}))
    return {
        "fwd": (lib.gdr_window_attn_fwd, [p, F, F, F, F, F, F, None, None, F, F, F, BIG, None], (1, 2, 3, 4, 5, 6, 9, 10),
                (1, 2, 3, 4, 5, 9)),
        "step": (lib.gdr_window_attn_step, [one, F, F, F, F, F, F, F, F, BIG, None], (1, 2, 3, 4, 5, 6, 7),
                 (1, 2, 3, 4, 5, 6, 7)),
        "bwd": (lib.gdr_window_attn_bwd, [p, F, F, F, F, F, F, None, None, F, F, F, F, BIG, None],
                (1, 2, 3, 4, 5, 6, 9, 10, 11), (1, 2, 3, 4, 5, 6, 9, 10, 11)),
    }


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 2), (dict(seq_len=-1), 2), (dict(num_seqs=-1), 2), (dict(num_q_heads=0), 2), (dict(num_q_heads=5), 2),
    (dict(num_kv_heads=0, k_stride=64, v_stride=64), 2), (dict(num_kv_heads=-2, num_q_heads=-4, q_stride=1, k_stride=1,
                                                               v_stride=1), 2),
    (dict(head_dim_qk=0), 2), (dict(head_dim_v=-1), 2), (dict(head_dim_qk=129), 4), (dict(head_dim_v=200), 4),
    (dict(window=0), 2), (dict(window=-3), 2), (dict(sinks=-1), 2), (dict(window=1 << 30, sinks=1 << 30), 2),
    (dict(scale=0.0), 2), (dict(scale=-1.0), 2), (dict(scale=float("inf")), 2), (dict(scale=float("nan")), 2),
    (dict(io_dtype=2), 3), (dict(io_dtype=0, out_dtype=1), 3), (dict(io_dtype=0, out_dtype=0, do_dtype=1), 3),
    (dict(grad_dtype=5), 3), (dict(q_stride=255), 2), (dict(k_stride=127), 2), (dict(v_stride=63), 2),
    (dict(q_stride=1 << 41), 2), (dict(batch=1 << 16, seq_len=1 << 16), 2),
    (dict(num_q_heads=1 << 16, num_kv_heads=1 << 16, head_dim_qk=128), 2),
])
@pytest.mark.parametrize("op", ["fwd", "step", "bwd"])
def test_problems(lib, op, kw, code):
    assert size(lib, op, attn(**kw))[0] == code
    assert lib.gdr_last_error_message()


def test_a_size_for_no_sequences(lib):
    """Tokens of no sequence are refused by the calls; the sizes are asked for before."""
    for op in ("fwd", "bwd"):
        assert size(lib, op, attn(io_dtype=0, out_dtype=0, do_dtype=0, batch=1, num_seqs=0, seq_len=100000))[0] == 0


def test_strides_of_prompts_and_steps(lib):
    """The tiles of prompts address a few tokens in 32 bits, single tokens are addressed in 64."""
    wide = attn(q_stride=1 << 30, k_stride=1 << 30, v_stride=1 << 30)
    assert size(lib, "fwd", wide)[0] == size(lib, "bwd", wide)[0] == 2 and size(lib, "step", wide)[0] == 0
    for name in ("fwd", "step", "bwd"):
        assert size(lib, name, attn())[0] == 0
        assert getattr(lib, "gdr_window_attn_%s_workspace_size" % name)(ctypes.byref(attn()), None) == 1
        assert getattr(lib, "gdr_window_attn_%s_workspace_size" % name)(None, ctypes.byref(ctypes.c_size_t())) == 1


@no_gpu
@pytest.mark.parametrize("name", ["fwd", "step", "bwd"])
def test_pointers(lib, name):
    fn, args, tensors, required = calls(lib)[name]
    for i in tensors:
        bad = list(args)
        bad[i] = ODD
        assert fn(*bad) == 2, (name, i)
    for i in required:
        bad = list(args)
        bad[i] = None
        assert fn(*bad) == 1, (name, i)
    bad = list(args)
    bad[0] = None
    assert fn(*bad) == 1


@no_gpu
def test_caches_come_together(lib):
    fn, args, _, _ = calls(lib)["fwd"]
    args[4] = args[5] = None
    assert fn(*args) == 1 and b"lens" in lib.gdr_last_error_message()          # lens without caches


@no_gpu
@pytest.mark.parametrize("name", ["fwd", "step", "bwd"])
def test_workspaces(lib, name):
    kw = dict(num_q_heads=1, num_kv_heads=1, batch=1, num_seqs=1, window=1 << 20, seq_len=32)
    fn, args, _, _ = calls(lib, **kw)[name]
    need = size(lib, name, attn(**{**kw, **({"seq_len": 1} if name == "step" else {})}))[1]
    assert need > 0
    at = len(args) - 3
    for ws, n in ((None, BIG), (ctypes.c_void_p((1 << 20) + 16), BIG), (FAKE, ctypes.c_size_t(need - 1))):
        bad = list(args)
        bad[at], bad[at + 1] = ws, n
        assert fn(*bad) == 6


@no_gpu
@pytest.mark.parametrize("name", ["fwd", "bwd"])
def test_sequence_offsets(lib, name):
    fn, args, _, _ = calls(lib, batch=1, num_seqs=2)[name]
    assert fn(*args) == 2                                # num_seqs differs from batch
    for offs in ([1, 5, 10], [0, 6, 5], [0, 4, 9], [0, 4, 11], [0, -1, 10]):
        t = torch.tensor(offs, dtype=torch.int32)
        bad = list(args)
        bad[7], bad[8] = FAKE, ctypes.c_void_p(t.data_ptr())
        assert fn(*bad) == 5, offs
    bad = list(args)
    bad[7] = FAKE                                        # one copy alone
    assert fn(*bad) == 1
    t = torch.tensor([0, 5, 10], dtype=torch.int32)
    bad = list(calls(lib)[name][1])
    bad[7], bad[8] = FAKE, ctypes.c_void_p(t.data_ptr())
    assert fn(*bad) == 5                                 # packed sequences take one batch row
    bad[7], bad[8] = ODD, ctypes.c_void_p(t.data_ptr())
    bad[0] = ctypes.byref(attn(batch=1, num_seqs=2))
    assert fn(*bad) == 2


@no_gpu
def test_step_takes_one_token(lib):
    fn, args, _, _ = calls(lib)["step"]
    for p in (attn(seq_len=2), attn(batch=1, seq_len=1), attn(seq_len=0)):
        assert fn(ctypes.byref(p), *args[1:]) == 2


@no_gpu
def test_nothing_to_do(lib):
    """No tokens: no pointers are needed, nothing is launched."""
    p = ctypes.byref(attn(seq_len=0))
    none = [None] * 8
    assert lib.gdr_window_attn_fwd(p, *none, None, None, None, ctypes.c_size_t(0), None) == 0
    assert lib.gdr_window_attn_bwd(p, *none, None, None, None, FAKE, BIG, None) == 0
    z = ctypes.byref(attn(batch=0, num_seqs=0, seq_len=1))
    assert lib.gdr_window_attn_step(z, *none, ctypes.c_size_t(0), None) == 0


def test_workspace_grows_with_the_tokens(lib):
    a, b = (size(lib, "bwd", attn(seq_len=n))[1] for n in (100, 10000))
    assert 0 < a < b
    assert size(lib, "bwd", attn(do_dtype=0))[1] > size(lib, "bwd", attn())[1]     # d_o in the io type


def test_binding_refuses(lib):
    q, k, v = torch.zeros(1, 8, 4, 16), torch.zeros(1, 8, 2, 16), torch.zeros(1, 8, 2, 16)
    cache, lens = (torch.zeros(1, 10, 2, 16), torch.zeros(1, 10, 2, 16)), torch.zeros(1, dtype=torch.int32)
    for f in (lambda: gdr.window_attn_fwd(q, k, v, 8), lambda: gdr.window_attn_step(q[:, 0], k[:, 0], v[:, 0], cache, lens, 8, 2),
              lambda: gdr.window_attn_bwd(q, k, v, q, q[..., 0], q, 8)):
        with pytest.raises(ValueError):                 # tensors on the CPU
            f()


def test_binding_checks(monkeypatch):
    """The binding's own checks, with the one for the device out of the way."""
    from chunkwise_gated_delta_local_amd import attn as m
    monkeypatch.setattr(m, "_device", lambda x: x.device)
    monkeypatch.setattr(m, "_launch", lambda *a: pytest.fail("launched"))
    q, k, v = torch.zeros(1, 8, 4, 16), torch.zeros(1, 8, 2, 16), torch.zeros(1, 8, 2, 24)
    cache, lens = (torch.zeros(1, 10, 2, 16), torch.zeros(1, 10, 2, 24)), torch.zeros(1, dtype=torch.int32)
    fwd = lambda q=q, k=k, v=v, w=8, s=2, **kw: m.window_attn_fwd(q, k, v, w, s, **kw)
    step = lambda q=q[:, 0], k=k[:, 0], v=v[:, 0], c=cache, n=lens, w=8, s=2, **kw: m.window_attn_step(q, k, v, c, n, w, s, **kw)
    o, lse = torch.zeros(1, 8, 4, 24), torch.zeros(1, 8, 4)
    bwd = lambda q=q, o=o, lse=lse, d=o, **kw: m.window_attn_bwd(q, k, v, o, lse, d, 8, 2, **kw)
    bad = [
        lambda: fwd(q=q[0]), lambda: fwd(k=k[0]), lambda: fwd(v=v[:, :7]), lambda: fwd(k=torch.zeros(1, 8, 2, 8)),
        lambda: fwd(k=k.to(torch.bfloat16)), lambda: fwd(v=torch.zeros(1, 8, 1, 24)), lambda: fwd(q=q[..., ::2], k=k[..., ::2]),
        lambda: fwd(q=q[:, :, :0]), lambda: fwd(w=0), lambda: fwd(s=-1), lambda: fwd(w=1 << 31), lambda: fwd(w=(1 << 31) - 2),
        lambda: fwd(scale=0.0), lambda: fwd(scale=float("inf")), lambda: fwd(scale=-0.1), lambda: fwd(lens=lens),
        lambda: fwd(cache=(cache[0],)), lambda: fwd(cache=(cache[0], None)), lambda: fwd(cache=(cache[0], cache[0])),
        lambda: fwd(cache=cache, s=3), lambda: fwd(cache=cache, lens=lens.long()), lambda: fwd(cache=cache, lens=torch.zeros(2, dtype=torch.int32)),
        lambda: fwd(cache=(cache[0].to(torch.bfloat16), cache[1])), lambda: fwd(out_dtype=torch.float16),
        lambda: fwd(cache=(cache[0].transpose(1, 2).contiguous().transpose(1, 2), cache[1])),
        lambda: step(q=q), lambda: step(c=None), lambda: step(n=None), lambda: step(n=lens.long()), lambda: step(w=9),
        lambda: step(k=k), lambda: bwd(o=o[..., :16]), lambda: bwd(lse=lse[..., :2]), lambda: bwd(d=o.half()),
        lambda: bwd(lse=lse.double()), lambda: bwd(grad_dtype=torch.float16), lambda: bwd(d=None), lambda: bwd(o=None), lambda: bwd(lse=None),
    ]
    for i, f in enumerate(bad):
        try:
            f()
        except (ValueError, TypeError):
            continue
        pytest.fail("call %d was taken" % i)


# ---------------------------------------------------------------- launches
CHILD = r"""
import ctypes, json, sys
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)           # before the library, so that its launches bind to it
sys.path[:0] = [sys.argv[2], sys.argv[2] + "/.."]
import test_attn_cpu as t
lib = t.api.load_library()
for name, kw in json.load(open(sys.argv[3])):
    fn, args, _, _ = t.calls(lib)[name]
    if kw.pop("packed", False):
        cu = (ctypes.c_int32 * (kw["num_seqs"] + 1))(*([0] * kw["num_seqs"] + [kw["seq_len"]]))
        args[7], args[8] = t.FAKE, ctypes.cast(cu, ctypes.c_void_p)
    p = t.attn(**kw)
    print("call", fn(ctypes.byref(p), *args[1:]), lib.gdr_last_error_message().decode(), flush=True)
"""


def test_launch_sizes(tmp_path):
    """From one token to 2^31 of them and from one head to a token of 2^22 elements: launches of at most 2^32 - 1 threads
    and 160 KB of LDS, or a refusal."""
    (tmp_path / "stand_in.cpp").write_text(STAND_IN)
    so = str(tmp_path / "stand_in.so")
    subprocess.check_call(["g++", "-O1", "-shared", "-fPIC", str(tmp_path / "stand_in.cpp"), "-o", so])
    most = (1 << 31) - 65
    shapes = [dict(batch=b, num_seqs=b, seq_len=t, num_q_heads=q, num_kv_heads=h, head_dim_qk=d, head_dim_v=d, window=w, sinks=s)
              for b, t in ((1, 1), (1, 100), (3, 5000), (1, most), (1 << 20, 2000), (most, 1))
              for q, h, d in ((1, 1, 1), (8, 2, 128), (64, 8, 64), (300, 1, 32), ((1 << 22) - 1, 1, 1), ((1 << 22) - 1, (1 << 22) - 1, 1))
              for w, s in ((1, 0), (128, 4), (1000, 1000), ((1 << 31) - 1, 0), (1, (1 << 31) - 2))]
    shapes += [dict(batch=1, num_seqs=n, seq_len=t, packed=True, num_q_heads=8, num_kv_heads=2, window=w, sinks=4)
               for n, t in ((1, 100), (1000, 100), (1 << 16, most), (1 << 16, 1 << 20)) for w in (16, 4096)]
    todo = []
    for io in (0, 1):
        for kw in shapes:
            kw = dict(kw, io_dtype=io, out_dtype=io, do_dtype=0)
            todo += [("fwd", kw), ("bwd", kw)]
            if not kw.get("packed"):
                todo.append(("step", dict(kw, seq_len=1)))
    (tmp_path / "todo.json").write_text(json.dumps(todo))
    out = subprocess.run([sys.executable, "-c", CHILD, so, HERE, str(tmp_path / "todo.json")], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    found, at, refused = [], 0, 0
    for line in out.stdout.splitlines():
        word = line.split()
        if word[0] == "launch":
            found.append(tuple(map(int, word[1:])))
            continue
        name, kw = todo[at]
        at += 1
        if int(word[1]):
            refused += 1
            heads = kw.get("num_q_heads", 4)
            assert int(word[1]) == 2 and "too large" in line and not found, (name, kw, line, found)
            # workgroups of at most 512 threads, none of them for less than a row: refused from 2^23 workgroups on
            assert kw["batch"] * kw["seq_len"] * heads > 1 << 22, (name, kw, line)
        else:
            assert found, (name, kw)
            for g, gyz, b, byz, lds in found:
                assert gyz == byz == 1 and 0 < b <= 1024 and 0 < g * b < 1 << 32 and lds <= 160 * 1024, (name, kw, found)
        found = []
    assert at == len(todo) and 0 < refused < len(todo) / 2


# ---------------------------------------------------------------- bookkeeping, compiled for the host
MODEL = r"""
#include <cstdint>
#include <cstdio>
#define __device__
#define __host__
#define __forceinline__ inline
%s
static void seq_range(const int32_t* cu, int n, int64_t, int64_t, int64_t* s, int64_t* e) { *s = cu[n]; *e = cu[n + 1]; }
// one lane that looks at 64 places for all
static int lane;
struct { struct { operator int() const { return lane; } } x; } threadIdx;
static int __builtin_popcll_(uint64_t x) { return __builtin_popcountll(x); }
#define __popcll __builtin_popcll_
#define __builtin_amdgcn_readfirstlane(x) (x)
%s
extern "C" {
// The keys that queries at positions first .. last see, in tiles of `tile` behind `skip` of them: position, row, cached
int keys_of(int first, int last, int len, int W, int S, int skip, int tile, int32_t* out) {
    Keys k(first, last, len, W, S);
    const int total = k.total();
    k.skip(skip);
    int m = 0;
    for (;;) {
        int pos, cnt, row; bool cached;
        k.next(tile, &pos, &cnt, &row, &cached);
        if (cnt == 0) break;
        for (int i = 0; i < cnt; ++i, ++m) { out[3 * m] = pos + i; out[3 * m + 1] = row + i; out[3 * m + 2] = cached; }
    }
    return m + skip == total ? m : -1;
}
int blocks_of(int batch, int T, int N, int packed, int TPB) { return (int)token_blocks(batch, T, N, packed, TPB); }
void rows_of(int rows, int G, int32_t* out) { RowBlock b = row_block(rows, G); out[0] = b.HPB; out[1] = b.TPB; out[2] = b.HC; }
int block_of(const int32_t* cu, int N, int T, int Ttot, int TPB, int b, int32_t* out) {
    Block x;
    if (!find_block(cu, N, T, Ttot, TPB, b, &x)) return 0;
    out[0] = x.n; out[1] = x.t0; out[2] = x.tn; out[3] = (int)x.start; out[4] = x.len;
    return 1;
}
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    src = open(os.path.join(CSRC, "gdr_attn.hpp")).read()
    cut = lambda a, b: src[src.index(a):src.index(b, src.index(a))]
    first = cut("struct RowBlock", "struct Block {")
    # the search over packed sequences: 64 lanes' answers one after the other
    block = cut("struct Block {", "// The keys that queries at")
    loop = re.search(r"const int step = .*?const int k = __popcll\(__ballot\(before\)\);", block, re.S).group(0)
    lanes = loop.replace("threadIdx.x & 63", "l").replace("const bool before =", "any |= (uint64_t)(")
    lanes = lanes.replace("const int step = (len + 63) / 64, i =", "const int i =")
    lanes = re.sub(r"(any \|= \(uint64_t\)\()(.*?);", r"\1\2) << l;", lanes, flags=re.S)
    lanes = lanes[:lanes.index("const int k =")]
    block = block.replace(loop, "const int step = (len + 63) / 64; uint64_t any = 0;\n"
                                "for (int l = 0; l < 64; ++l) { %s }\nconst int k = __popcll(any);" % lanes)
    keys = cut("struct Keys {", "// ------")
    d = tmp_path_factory.mktemp("model")
    (d / "m.cpp").write_text(MODEL % (first, block + keys))
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-shared", "-fPIC",
                           str(d / "m.cpp"), "-o", str(d / "m.so")])
    return ctypes.CDLL(str(d / "m.so"))


def seen(first, last, len_, W, S):
    """Every key that some query of the block sees, its row and whether it is cached"""
    res = {}
    for j in range(last + 1):
        if any(j <= p and (p - j < W or j < S) for p in range(first, last + 1)):
            res[j] = (j - len_, 0) if j >= len_ else (j if j < S else S + (j - S) % W, 1)
    return res


def test_keys_of_a_block(model):
    rnd = random.Random(5)
    out = (ctypes.c_int32 * 3000)()
    grid = [(w, s, n, f, l) for w in (1, 2, 5, 8) for s in (0, 1, 3, 9) for n in (0, 1, 2, 5, 8, 9, 12, 17, 30)
            for f in (0, 1, 4, 9) for l in (0, 3, 7)]
    grid += [(rnd.randint(1, 70), rnd.choice([0, 0, 1, 4, 40]), rnd.randint(0, 150), rnd.randint(0, 100), rnd.randint(0, 40))
             for _ in range(400)]
    for W, S, n, f, l in grid:
        first, last = n + f, n + f + l
        want = seen(first, last, n, W, S)
        for tile in (1, 32):
            m = model.keys_of(first, last, n, W, S, 0, tile, out)
            assert m == len(want), (W, S, n, f, l, m)
            got = {out[3 * i]: (out[3 * i + 1], out[3 * i + 2]) for i in range(m)}
            assert got == want, (W, S, n, f, l)
        for skip in {0, 1, len(want) // 2, len(want) - 1, len(want)}:
            order = [out[3 * i] for i in range(model.keys_of(first, last, n, W, S, 0, 7, out))]
            m = model.keys_of(first, last, n, W, S, skip, 7, out)
            assert [out[3 * i] for i in range(m)] == order[skip:], (W, S, n, f, l, skip)


def test_keys_near_the_largest_positions(model):
    """Positions up to 2^31 - 1: no sum in the bookkeeping overflows."""
    out = (ctypes.c_int32 * 3000)()
    top = (1 << 31) - 1
    for W, S, n, last in ((4, 2, top - 10, top - 1), (4, 2, top - 1, top - 1), (7, 0, top - 20, top - 5)):
        m = model.keys_of(n, last, n, W, S, 0, 32, out)
        lo = max(n - W + 1, S)
        want = {j: (j, 1) for j in range(min(S, n))}
        want.update({j: (S + (j - S) % W, 1) if j < n else (j - n, 0) for j in range(lo, last + 1)})
        assert {out[3 * i]: (out[3 * i + 1], out[3 * i + 2]) for i in range(m)} == want
    for W, S in ((top, 0), (1, top - 1), (top - 5, 5)):                        # a window or sinks beyond all tokens
        m = model.keys_of(3, 20, 3, W, S, 0, 32, out)
        assert sorted(out[3 * i] for i in range(m)) == list(range(21))


def test_every_token_lies_in_one_block(model):
    rnd = random.Random(6)
    out = (ctypes.c_int32 * 5)()
    cases = [[0], [1], [0, 0, 5], [31, 32, 33], [0, 64, 0, 1], [1] * 200, [0] * 130 + [7] + [0] * 70]
    cases += [[rnd.choice([0, 1, 2, rnd.randint(0, 80)]) for _ in range(rnd.randint(1, 300))] for _ in range(60)]
    for lens in cases:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        T, N = cu[-1], len(lens)
        host = (ctypes.c_int32 * (N + 1))(*cu)
        for TPB in (1, 5, 32, 128):
            at = []
            for b in range(model.blocks_of(1, T, N, 1, TPB)):
                if model.block_of(host, N, T, T, TPB, b, out):
                    n, t0, tn, start, ln = out
                    assert start == cu[n] and ln == lens[n] and 0 < tn <= TPB and t0 % TPB == 0
                    at += [start + t0 + i for i in range(tn)]
            assert sorted(at) == list(range(T)), (lens, TPB)
    for B, T, TPB in ((1, 1, 32), (3, 33, 32), (4, 128, 128), (2, 7, 5)):
        at = []
        for b in range(model.blocks_of(B, T, B, 0, TPB)):
            assert model.block_of(None, B, T, B * T, TPB, b, out)
            n, t0, tn, start, ln = out
            at += [start + t0 + i for i in range(tn)]
        assert sorted(at) == list(range(B * T))


def test_rows_of_a_block(model):
    out = (ctypes.c_int32 * 3)()
    for rows in (32, 128):
        for G in (1, 2, 3, 5, 8, 31, 32, 33, 64, 100, 128, 300):
            model.rows_of(rows, G, out)
            heads, tokens, blocks = out
            assert heads * tokens <= rows and tokens >= 1 and (blocks - 1) * heads < G <= blocks * heads
            for r in range(heads * tokens):                # the division by multiplication that the kernels make
                assert (r * ((65536 + heads - 1) // heads)) >> 16 == r // heads


# ---------------------------------------------------------------- the bounds notice mistakes
MISTAKES = {
    "window one longer": lambda p, j, W, S: (j <= p) & ((p - j < W + 1) | (j < S)),
    "window one shorter": lambda p, j, W, S: (j <= p) & ((p - j < max(W - 1, 1)) | (j < S)),
    "one sink less": lambda p, j, W, S: (j <= p) & ((p - j < W) | (j < S - 1)),
    "sinks of the first tokens alone": lambda p, j, W, S: (j <= p) & ((p - j < W) | ((j < S) & (p < 2 * W))),
    "a token ahead": lambda p, j, W, S: (j <= p + 1) & ((p - j < W) | (j < S)),
    "not itself": lambda p, j, W, S: ((j < p) | (j == 0)) & ((p - j < W) | (j < S)),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mistake", sorted(MISTAKES))
def test_bounds_notice_a_wrong_mask(monkeypatch, mistake, dtype):
    import numpy as np
    import attn_common as ac
    c = ac.attn_case(dtype, [70, 23], 4, 2, 32, 24, 12, 2, seed=3)
    o, lse, eo, el, _ = ac.forward_reference(c)
    grads = ac.backward_reference(c, o, lse)
    monkeypatch.setattr(ac.oa, "sees", MISTAKES[mistake])
    o2, lse2 = ac.forward_reference(c)[:2]
    half = torch.finfo(c["q"].dtype).eps / 2
    assert (np.abs(o2 - o) > 4 * (eo + half * np.abs(o))).any() and (np.abs(lse2 - lse) > 4 * el).any()
    wrong = ac.backward_reference(c, o, lse)
    for name, (g, e) in grads.items():
        assert (np.abs(wrong[name][0] - g) > 4 * (e + half * np.abs(g))).any(), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_notice_a_lost_key_and_a_wrong_head(dtype):
    """A key that is left out of one row, a tile's sums that are not rescaled, a neighbour's key head."""
    import numpy as np
    import attn_common as ac
    c = ac.attn_case(dtype, [90], 4, 2, 32, 32, 64, 1, seed=4)
    o, lse, eo, el, _ = ac.forward_reference(c)
    half = torch.finfo(c["q"].dtype).eps / 2
    q, k, v = ac.f64(c["q"])[0], ac.f64(c["k"])[0], ac.f64(c["v"])[0]
    at = np.arange(90)
    _, _, p = ac.oa.attend(q[:, 0], k[:, 0], v[:, 0], at, at, 64, 1, c["scale"])
    limit = 4 * (eo[:, 0] + half * np.abs(o[:, 0]))
    lost = p.copy()
    lost[89, 60] = 0
    assert (np.abs(lost @ v[:, 0] - o[:, 0])[89] > limit[89]).any()
    part = p.copy()
    part[:, :32] *= 2.0                                  # the reference moved by one in the exponent
    assert (np.abs((part / part.sum(1, keepdims=True)) @ v[:, 0] - o[:, 0]) > limit).any()
    assert (np.abs(p @ v[:, 1] - o[:, 0]) > limit).any()
