"""Chunked gated delta-rule forward for AMD MI355X (gfx950), and the operators
that stand next to it in a layer: the short causal convolution, the selective
state space scan, the norms (layer norm, the gated RMS norm, the residual sum
with its norms) and attention with a sliding window and sinks.

The compute path is a C-ABI shared library (``libgdr.so``, built from
``csrc/``) of hand-written HIP kernels; this package only marshals torch
tensors into it. Importing the package does not load the library; the first
call does, and fails loudly if the library is missing.
"""
from .api import Forward, chunk_fwd, chunk_fwd_debug, recurrent_fwd, workspace_size, validate  # noqa: F401
from .mixer import (conv_bwd, conv_fwd, conv_step, gated_norm_bwd, gated_norm_fwd, layer_norm_bwd,  # noqa: F401
                    layer_norm_fwd, residual_norm_bwd, residual_norm_fwd, scan_bwd, scan_fwd, scan_step)
from .attn import window_attn_bwd, window_attn_fwd, window_attn_step  # noqa: F401
