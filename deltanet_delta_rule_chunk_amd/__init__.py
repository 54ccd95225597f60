"""MI355X (gfx950) DeltaNet delta-rule forward and decode step, and the gated
linear recurrence and q / k maps beside it.

The computation lives in hand-written HIP kernels behind the C ABI of
``libdeltanet.so`` (include/deltanet.h); ``binding`` marshals PyTorch tensors
to it.  The library is loaded on first use and its absence is an error.
"""

from .binding import (chunk_fwd, decode_step, delta_rule, linear_chunk_bwd,  # noqa: F401
                      linear_chunk_fwd, linear_decode_step, linear_rule, load, qk_norm_rope,
                      qk_norm_rope_bwd, rotary_qk, workspace_bytes)

__all__ = ["chunk_fwd", "decode_step", "delta_rule", "linear_chunk_bwd", "linear_chunk_fwd",
           "linear_decode_step", "linear_rule", "load", "qk_norm_rope", "qk_norm_rope_bwd",
           "rotary_qk", "workspace_bytes"]
