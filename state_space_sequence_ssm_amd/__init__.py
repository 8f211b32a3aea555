"""Mamba-3 SSM core on AMD MI355X (gfx950): hand-written HIP kernels behind a
C ABI (libm3ssm.so, include/m3ssm.h) with a thin torch binding.

Entry points (same names as the C ABI):
  m3_ssm_prefill        chunked prefill over whole sequences
  m3_ssm_decode_step    one token against a resident fp32 state
  m3_rope_angles_cumsum cumulative rotation angles
  m3_causal_conv, m3_causal_conv_step, m3_causal_conv_backward
                        short causal convolution in front of the core
  m3_selective_scan, m3_selective_scan_step, m3_selective_scan_backward
                        selective scan with a decay per channel and state
  m3_gated_norm, m3_gated_norm_backward
                        gated group RMS norm behind the core
  m3_residual_norm, m3_residual_norm_backward
                        residual sum and RMS norm in front of the next block
  m3_linear_attention, m3_linear_attention_step, m3_linear_attention_backward
                        linear attention with a constant decay for each head
  m3_qk_norm_rope, m3_qk_norm_rope_backward
                        norm of queries and keys for each head, and their rotation
Outputs carry no gradient history; gradients come from the `_backward` entry points.
"""
from ._lib import LAYER_CALLS, LIB_PATH, MIXER_CALLS, load  # noqa: F401

__version__ = "0.1.0"


def __getattr__(name):
    # the torch binding is imported lazily so that the ctypes layer can be
    # used (and tested) without initialising a GPU runtime
    if name in ("m3_ssm_prefill", "m3_ssm_decode_step", "m3_rope_angles_cumsum", "M3Error") or name in LAYER_CALLS \
            or name in MIXER_CALLS:
        from . import ops
        return getattr(ops, name)
    raise AttributeError(name)
