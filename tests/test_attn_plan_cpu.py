"""How the window attention's forward pass is shared out, from the launches that a call makes (written down by stand-ins
for HIP's launch): by the keys that a query can see, which are no more than its sequence has where nothing is cached."""
import json
import os
import subprocess
import sys

import pytest
import torch

from test_launch_sizes_cpu import STAND_IN

HERE = os.path.dirname(os.path.abspath(__file__))
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="replaces the launch of kernels")

CHILD = r"""
import ctypes, json, sys
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)           # before the library, so that its launches bind to it
sys.path[:0] = [sys.argv[2], sys.argv[2] + "/.."]
import test_attn_cpu as t
lib = t.api.load_library()
for cached, kw in json.loads(sys.argv[3]):
    p, F = t.attn(**kw), t.FAKE
    c = (F if cached else None, F if cached else None, F if cached == 2 else None)
    need = ctypes.c_size_t(t.size(lib, "fwd", p)[1])
    print("call", lib.gdr_window_attn_fwd(ctypes.byref(p), F, F, F, *c, None, None, F, F, F, need, None), need.value, flush=True)
"""


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "stand_in.cpp").write_text(STAND_IN)
    so = str(d / "stand_in.so")
    subprocess.check_call(["g++", "-O1", "-shared", "-fPIC", str(d / "stand_in.cpp"), "-o", so])

    def run(calls):
        """[(workspace, [workgroups of every launch])]; a call: (0 no caches, 1 empty ones, 2 with lens; problem)"""
        out = subprocess.run([sys.executable, "-c", CHILD, so, HERE, json.dumps(calls)], capture_output=True, text=True, timeout=120)
        assert out.returncode == 0, out.stderr[-2000:]
        res, grids = [], []
        for line in out.stdout.splitlines():
            w = line.split()
            if w[0] == "launch":
                grids.append(int(w[1]))
            else:
                assert w[1] == "0", line
                res.append((int(w[2]), grids))
                grids = []
        assert len(res) == len(calls)
        return res
    return run


def problem(io, **kw):
    return dict(dict(io_dtype=io, out_dtype=io, do_dtype=0, sinks=0, head_dim_qk=64, head_dim_v=64), **kw)


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("batch,seq_len,heads", [(1, 512, 1), (1, 512, 4), (3, 200, 2), (1, 2048, 1), (100, 64, 7)])
def test_a_window_beyond_the_sequence_changes_nothing(launches, io, batch, seq_len, heads):
    kw = dict(batch=batch, num_seqs=batch, seq_len=seq_len, num_q_heads=heads, num_kv_heads=heads)
    windows = (seq_len, seq_len + 1, 65536, (1 << 31) - 1)
    found = launches([(cached, problem(io, window=w, **kw)) for cached in (0, 1) for w in windows])
    for same in (found[:4], found[4:]):
        assert all(g == same[0][1] for _, g in same), found


def test_cached_pieces_count_the_keys_behind_them(launches):
    """700 blocks of 32 rows, fp32. Over a window of 4,096 each walks 128 tiles and more of the caches, which pays for sharing
    them among a workgroup's wavefronts; without caches two tiles do not."""
    kw = problem(0, batch=350, num_seqs=350, seq_len=64, num_q_heads=1, num_kv_heads=1, window=4096)
    (_, cached), (_, alone) = launches([(2, kw), (0, kw)])
    assert cached[0] == 700 and alone[0] == 352


@pytest.mark.parametrize("io", [0, 1])
def test_the_workspace_does_for_either(launches, io):
    """With the size that is asked for before the caches are known, whatever is launched has room for its parts."""
    shapes = [problem(io, batch=b, num_seqs=b, seq_len=t, num_q_heads=q, num_kv_heads=k, window=w)
              for b, t in ((1, 1), (1, 40), (1, 700), (5, 33), (2, 5000)) for q, k in ((1, 1), (8, 2), (3, 3))
              for w in (16, 1000, 40000, (1 << 31) - 1)]
    shared = 0
    calls = [(c, kw) for kw in shapes for c in (0, 1, 2)]
    for (_, kw), (have, grids) in zip(calls, launches(calls)):
        rows = kw["batch"] * kw["seq_len"] * kw["num_q_heads"]
        per = 32 // (kw["num_q_heads"] // kw["num_kv_heads"])                 # tokens of a block
        work = kw["batch"] * -(-kw["seq_len"] // per) * kw["num_kv_heads"]
        if len(grids) > 1 and grids[1] == (rows + 3) // 4 and grids[0] % work == 0 and grids[0] > work:
            shared += 1
            assert have >= grids[0] // work * rows * (kw["head_dim_v"] + 2) * 4, (kw, grids, have)
    assert shared > 0
