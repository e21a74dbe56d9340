"""Limits of the layer operators' arguments, found on the host: calls of no sequence or row, which pass every check and
launch nothing."""
import ctypes

import pytest

from chunkwise_gated_delta_local_amd import api
from test_mixer_cpu import scan

FAKE = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def lib():
    return api.load_library()


@pytest.mark.parametrize("name", ["x_stride", "dt_stride", "z_stride", "b_stride", "c_stride"])
def test_token_strides_of_the_scan(lib, name):
    """One token of every sequence is indexed in 64 bits: only the tiles of scan_fwd and scan_bwd end at 2^22."""
    F = FAKE
    for stride, tiles in (((1 << 22) - 1, 0), (1 << 22, 2), (1 << 39, 2)):
        none = dict(batch=0, num_seqs=0, **{name: stride})
        p = ctypes.byref(scan(seq_len=1, **none))
        assert lib.gdr_scan_step(p, F, F, F, F, F, F, F, F, F, F, None) == 0, stride
        p = ctypes.byref(scan(seq_len=10, **none))
        assert lib.gdr_scan_fwd(p, F, F, F, F, F, F, F, F, F, None, None, F, F, None, 0, None) == tiles, stride
    p = ctypes.byref(scan(seq_len=1, batch=0, num_seqs=0, **{name: 31}))
    assert lib.gdr_scan_step(p, F, F, F, F, F, F, F, F, F, F, None) == 2
