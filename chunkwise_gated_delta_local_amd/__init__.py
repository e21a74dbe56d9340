"""Chunked gated delta-rule forward for AMD MI355X (gfx950), and the operators
that stand next to it in a layer: the short causal convolution, the selective
state space scan and layer norm.

The compute path is a C-ABI shared library (``libgdr.so``, built from
``csrc/``) of hand-written HIP kernels; this package only marshals torch
tensors into it. Importing the package does not load the library; the first
call does, and fails loudly if the library is missing.
"""
from .api import Forward, chunk_fwd, chunk_fwd_debug, recurrent_fwd, workspace_size, validate  # noqa: F401
from .mixer import (conv_bwd, conv_fwd, conv_step, layer_norm_bwd, layer_norm_fwd, scan_bwd, scan_fwd,  # noqa: F401
                    scan_step)
