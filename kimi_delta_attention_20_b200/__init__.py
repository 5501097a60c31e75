"""Kimi Delta Attention (KDA) for NVIDIA B200 (sm_100a).

`chunk_kda` (chunkwise forward, with autograd through `chunk_kda_bwd`), `recurrent_step` (one decode token per
sequence, state updated in place) and `decode_token` (the serving token: conv
update + SiLU, the recurrent step and the output gate in one launch) call the
C-ABI library libkda.so built from csrc/
(`python -m kimi_delta_attention_20_b200.build`).

Around the state update of a layer: `rms_norm` (residual, output gate; `rms_norm_quant`
with an 8-bit output), `causal_conv` (short convolution + SiLU over sequences) and
`chunk_gated_scan` (elementwise gated recurrence), with gradients and single-token forms.
"""
from .layer_ops import (causal_conv, causal_conv_bwd, causal_conv_step, chunk_gated_scan,  # noqa: F401
                        chunk_gated_scan_bwd, gated_scan_step, rms_norm, rms_norm_bwd, rms_norm_quant)
from .ops import chunk_bwd_workspace_bytes, chunk_kda, chunk_kda_bwd, chunk_workspace_bytes, decode_token, recurrent_step  # noqa: F401

__all__ = ["chunk_kda", "chunk_kda_bwd", "recurrent_step", "decode_token", "chunk_workspace_bytes",
           "chunk_bwd_workspace_bytes", "rms_norm", "rms_norm_quant", "rms_norm_bwd", "causal_conv",
           "causal_conv_step", "causal_conv_bwd", "chunk_gated_scan", "gated_scan_step", "chunk_gated_scan_bwd"]
