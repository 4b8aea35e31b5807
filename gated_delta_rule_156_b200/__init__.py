"""Kimi Delta Attention (KDA) and the operators around it for B200 (sm_100a).

The kernels live in the in-tree ``libkda.so`` (sources under ``csrc/``, public
C ABI in ``include/kda.h`` and ``include/kda_layer.h``); this package only
marshals torch tensors into that ABI.
"""
from .kda import (KdaError, KdaShape, block_norm_bwd, block_norm_fwd,  # noqa: F401
                  chunk_fwd, library, library_path, recurrent_step,
                  short_conv_bwd, short_conv_fwd, short_conv_step,
                  ssm_scan_bwd, ssm_scan_fwd, ssm_step)

__all__ = ["chunk_fwd", "recurrent_step", "short_conv_fwd", "short_conv_bwd",
           "short_conv_step", "ssm_scan_fwd", "ssm_scan_bwd", "ssm_step",
           "block_norm_fwd", "block_norm_bwd", "library", "library_path",
           "KdaError", "KdaShape"]
