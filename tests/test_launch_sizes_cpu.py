"""Launch sizes of the layer operators at the largest problems they take. A child process binds the library to stand-ins
for HIP's launch that write down grid, block and LDS of every launch and start nothing, so that no device and no
memory is needed: HIP counts the threads of a launch in 32 bits."""
import ctypes
import json
import os
import subprocess
import sys

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="replaces the launch of kernels")

STAND_IN = r"""
#include <cstddef>
#include <cstdint>
#include <cstdio>
struct Dim { uint32_t x, y, z; };
static Dim grid, block;
static size_t bytes;
extern "C" {
int __hipPushCallConfiguration(Dim g, Dim b, size_t lds, void*) {
    grid = g; block = b; bytes = lds;
    return 0;
}
int __hipPopCallConfiguration(Dim* g, Dim* b, size_t* lds, void**) {
    *g = grid; *b = block; *lds = bytes;
    return 0;
}
int hipLaunchKernel(const void*, Dim g, Dim b, void**, size_t lds, void*) {
    printf("launch %u %u %u %u %zu\n", g.x, g.y * g.z, b.x, b.y * b.z, lds);
    fflush(stdout);
    return 0;
}
int hipGetLastError() { return 0; }
}
"""

CHILD = r"""
import ctypes, json, sys
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)           # before the library, so that its launches bind to it
sys.path[:0] = [sys.argv[2], sys.argv[2] + "/.."]
import test_mixer_cpu as t
lib = t.api.load_library()
for name, kw in json.loads(sys.argv[3]):
    fn, args, _, _ = t.calls(lib)[name]
    p = t.norm(**kw) if "norm" in name else (t.conv if "conv" in name else t.scan)(**kw)
    print("call", fn(ctypes.byref(p), *args[1:]), lib.gdr_last_error_message().decode(), flush=True)
"""


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    d = tmp_path_factory.mktemp("launch")
    (d / "stand_in.cpp").write_text(STAND_IN)
    so = str(d / "stand_in.so")
    subprocess.check_call(["g++", "-O1", "-shared", "-fPIC", str(d / "stand_in.cpp"), "-o", so])

    def run(calls):
        """[(status, message, [(workgroups, threads, lds)])] of each call"""
        out = subprocess.run([sys.executable, "-c", CHILD, so, HERE, json.dumps(calls)], capture_output=True, text=True,
                             timeout=120)
        assert out.returncode == 0, out.stderr[-2000:]
        res, now = [], []
        for line in out.stdout.splitlines():
            word = line.split()
            if word[0] == "launch":
                g, gyz, b, byz, lds = map(int, word[1:])
                assert gyz == byz == 1
                now.append((g, b, lds))
            else:
                res.append((int(word[1]), " ".join(word[2:]), now))
                now = []
        assert len(res) == len(calls)
        return res
    return run


def test_norm_rows(launches):
    """Rows go round the grid, so that any number of them is taken."""
    calls = [(op, dict(rows=r, cols=c, x_stride=c, io_dtype=io, out_dtype=io, dy_dtype=io, grad_dtype=io))
             for op in ("layer_norm_fwd", "layer_norm_bwd") for io in (0, 1)
             for r, c in ((256, 4096), (1 << 21, 128), ((1 << 26) + 3, 5000), (1 << 28, 136), ((1 << 28) + 1, 1024),
                          ((1 << 30) + 37, 2), (1 << 38, 64), (1 << 40, 1), (1 << 40, 16384))]
    for (op, kw), (status, message, found) in zip(calls, launches(calls)):
        assert status == 0, (op, kw, message)
        assert found and all(0 < g * b < 1 << 32 for g, b, _ in found), (op, kw, found)


def test_conv_channels(launches):
    """Channels are counted in an int, several to a lane: more than 2^30 of them are refused."""
    calls = [(op, dict(batch=1, num_seqs=1, seq_len=1, channels=D, x_stride=D, width=W))
             for op in ("conv_fwd", "conv_step", "conv_bwd") for W in (2, 4)
             for D in (1, 5, 8192, (1 << 22) + 3, 1 << 30, (1 << 30) + 1, (1 << 31) - 512, (1 << 31) - 2, (1 << 31) - 1)]
    for (op, kw), (status, message, found) in zip(calls, launches(calls)):
        D = kw["channels"]
        assert status == (2 if D > 1 << 30 else 0), (op, kw, message)
        if status:
            assert not found and "channels" in message, (op, kw, message, found)
        else:
            assert found and all(0 < b <= 1024 and 0 < g * b < 1 << 32 for g, b, _ in found), (op, kw, found)
            assert found[0][0] * found[0][1] * 8 >= D, (op, kw, found)     # a lane takes 8 channels at most


def test_scan_sizes(launches):
    """From one token to 2^30 sequences and the widest rows: a launch within HIP's limits and a compute unit's LDS, or a
    refusal."""
    most = (1 << 22) - 1
    shapes = [(1, 1, 1, 1), (1, 1, most, 1), (1, 300, most, 1), (1, 1, 1 << 21, 1 << 21), (1, 65536, 4096, 1),
              (1, (1 << 31) - 65, 16, 1), (1 << 22, 100, 64, 4), (1 << 30, 1, 1, 1), (1 << 20, 1, 4096, 2), (3, 0, 64, 1),
              (13, 4099, 1540, 4), (2, 700, 1536, 1)]
    calls = [(op, dict(batch=b, num_seqs=b, seq_len=1 if op == "scan_step" else t, channels=D, groups=G, state_dim=S,
                       x_stride=D, dt_stride=D, z_stride=D, b_stride=G * S, c_stride=G * S))
             for op in ("scan_step", "scan_bwd") for b, t, D, G in shapes for S in (1, 8, 16, 24, 32, 64) if G * S <= most]
    refused = 0
    for (op, kw), (status, message, found) in zip(calls, launches(calls)):
        if status:
            refused += 1
            N, D, G, S = (kw[k] for k in ("batch", "channels", "groups", "state_dim"))
            assert status == 2 and "too large" in message and not found, (op, kw, status, message)
            # lanes of the single tokens: 4 states each, a power of two to a channel; of the tiles: at most 8 wavefronts to
            # 16 channels, whose workgroups come in fours
            lanes = N * D * 2 * -(-S // 4) if op == "scan_step" else N * G * -(-(D // G) // 64) * 4 * 512
            assert lanes >= 1 << 32, (op, kw)
        else:
            assert found and all(0 < b <= 1024 and 0 < g * b < 1 << 32 and lds <= 160 * 1024 for g, b, lds in found), (op, kw)
    assert 0 < refused < len(calls) / 2
