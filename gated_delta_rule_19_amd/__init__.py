"""Kimi Delta Attention (KDA) for AMD MI355X (gfx950).

The computation lives in ``libkda.so`` (hand-written HIP kernels behind the C
ABI of ``include/kda.h``); this package is its thin Python binding.  The
library is loaded on first use and every call raises if it is missing.
"""
from ._block import (beam_select, block_norm, decay_attention, decay_attention_step,
                     state_reorder)
from ._native import (CHUNK, HEAD_DIM, KDA_BF16, KDA_F32, KdaError, LIB_PATH, chunk_prefill,
                      chunk_prefill_checkpoint, chunk_prefill_checkpoints, chunk_prefill_gated,
                      decode_replay, decode_replay_gated, decode_step, decode_step_gated, load, plan_num_segments, prefill_workspace_size,
                      segment_scan, segment_transition, status_string, version)
from ._recurrent import (selective_scan, selective_scan_step, short_conv, short_conv_step,
                         state_load, state_store)

__all__ = [
    "CHUNK", "HEAD_DIM", "KDA_BF16", "KDA_F32", "KdaError", "LIB_PATH", "beam_select", "block_norm", "chunk_prefill", "chunk_prefill_checkpoint",
    "chunk_prefill_checkpoints", "chunk_prefill_gated", "decay_attention", "decay_attention_step",
    "decode_replay", "decode_replay_gated", "decode_step", "decode_step_gated", "load", "plan_num_segments", "prefill_workspace_size", "segment_scan", "segment_transition",
    "selective_scan", "selective_scan_step", "short_conv", "short_conv_step", "state_load", "state_reorder", "state_store",
    "status_string", "version",
]
