"""MI355X (gfx950) Mamba2 causal conv1d + SSD chunked scan with segment-local state passing.

Around the scan: its single-token form, linear attention with a decay per head, the gated
delta rule, the gated group norm of a mixer's output, the norms around a block and rotary
positions.

The compute path is libssd.so (hand-written HIP for CDNA4, C ABI in
include/ssd.h, ssd_mixer.h and ssd_layer.h).  This package only marshals torch tensors into that ABI.
"""
from ._lib import (SSD_BF16, SSD_F32, SSD_GATE_LINEAR, SSD_GATE_NONE, SSD_GATE_SIGMOID,
                   SSD_GATE_SILU, SSD_ROPE_HALF, SSD_ROPE_INTERLEAVED,
                   SSD_NORM_AFTER, SSD_NORM_BEFORE, SSD_NORM_NONE,
                   SSD_NORM_SILU, SSD_WS_BACKWARD, SSD_WS_FORWARD,
                   SSD_WS_FORWARD_CONV, SSDError, load)
from .layer import (BlockNormBackwardBuffers, GatedDeltaBackwardBuffers, GatedDeltaForwardBuffers,
                    block_norm_backward, block_norm_forward, gdelta_backward, gdelta_forward,
                    make_block_norm, make_gdelta, make_rope, rope_backward, rope_forward,
                    rope_frequencies, ssd_block_norm_bwd, ssd_block_norm_fwd,
                    ssd_block_norm_workspace_bytes, ssd_gdelta_bwd, ssd_gdelta_fwd, ssd_gdelta_step,
                    ssd_gdelta_workspace_bytes, ssd_rope)
from .mixer import (LinAttnBackwardBuffers, LinAttnForwardBuffers, NormBackwardBuffers,
                    StepState, linattn_backward, linattn_forward, make_linattn, make_norm,
                    norm_backward, norm_forward, ssd_linattn_bwd, ssd_linattn_fwd,
                    ssd_linattn_step, ssd_linattn_workspace_bytes, ssd_norm_bwd, ssd_norm_fwd,
                    ssd_norm_workspace_bytes, ssd_token_step)
from .ops import (BackwardBuffers, ForwardBuffers, Segments, backward, forward, make_problem,
                  ssd_apply_init_state, ssd_boundary_scan, ssd_conv1d_bwd, ssd_conv1d_fwd,
                  ssd_conv_segment_output, ssd_conv_segment_states,
                  ssd_segment_bwd, ssd_segment_bwd_chunks, ssd_segment_bwd_pass,
                  ssd_segment_bwd_summary,
                  ssd_segment_fwd, ssd_segment_fwd_noalloc, ssd_segment_output, ssd_segment_output_fused,
                  ssd_segment_states, ssd_workspace_bytes, summary_numel)

__all__ = ["SSD_BF16", "SSD_F32", "SSD_NORM_AFTER", "SSD_NORM_BEFORE", "SSD_NORM_NONE",
           "SSD_NORM_SILU", "LinAttnBackwardBuffers", "LinAttnForwardBuffers",
           "NormBackwardBuffers", "StepState", "linattn_backward", "linattn_forward",
           "make_linattn", "make_norm", "norm_backward", "norm_forward", "ssd_linattn_bwd",
           "ssd_linattn_fwd", "ssd_linattn_step", "ssd_linattn_workspace_bytes", "ssd_norm_bwd",
           "ssd_norm_fwd", "ssd_norm_workspace_bytes", "ssd_token_step",
           "SSD_GATE_LINEAR", "SSD_GATE_NONE", "SSD_GATE_SIGMOID", "SSD_GATE_SILU", "SSD_ROPE_HALF",
           "SSD_ROPE_INTERLEAVED", "BlockNormBackwardBuffers", "GatedDeltaBackwardBuffers",
           "GatedDeltaForwardBuffers", "block_norm_backward", "block_norm_forward", "gdelta_backward",
           "gdelta_forward", "make_block_norm", "make_gdelta", "make_rope", "rope_backward",
           "rope_forward", "rope_frequencies", "ssd_block_norm_bwd", "ssd_block_norm_fwd",
           "ssd_block_norm_workspace_bytes", "ssd_gdelta_bwd", "ssd_gdelta_fwd", "ssd_gdelta_step",
           "ssd_gdelta_workspace_bytes", "ssd_rope",
           "SSD_WS_BACKWARD", "SSD_WS_FORWARD", "SSD_WS_FORWARD_CONV",
           "SSDError", "load",
           "BackwardBuffers", "ForwardBuffers", "Segments", "backward", "forward",
           "make_problem", "ssd_apply_init_state", "ssd_boundary_scan", "ssd_conv1d_bwd",
           "ssd_conv1d_fwd", "ssd_conv_segment_output", "ssd_conv_segment_states",
           "ssd_segment_bwd", "ssd_segment_bwd_chunks", "ssd_segment_bwd_pass",
           "ssd_segment_bwd_summary", "ssd_segment_fwd", "ssd_segment_fwd_noalloc", "ssd_segment_output",
           "ssd_segment_output_fused", "ssd_segment_states", "ssd_workspace_bytes", "summary_numel"]
