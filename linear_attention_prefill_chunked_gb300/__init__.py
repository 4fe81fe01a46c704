"""GB300 (sm_103a) chunked KDA prefill and decode, and the operators of the layers around them.

The compute lives in ``libkda_gb300.so`` (hand-written CUDA kernels behind the
C ABI of ``include/kda.h``); this package is its thin binding.
"""
from .api import (KdaDesc, KdaError, chunk_prefill, chunk_prefill_act, decode, decode_draft, load,
                  make_desc, prefill_min_workspace_size, prefill_path, prefill_workspace_size,
                  read_device_status)
from .layer import (causal_conv, causal_conv_backward, causal_conv_decode, causal_conv_draft, commit_draft,
                    gated_decode, gated_decode_draft, gated_scan, gated_scan_backward, sample,
                    sample_probs, ssm_decode,
                    ssm_decode_draft, ssm_scan, ssm_scan_workspace_size, verify_draft)

__all__ = ["KdaDesc", "KdaError", "chunk_prefill", "chunk_prefill_act", "decode", "decode_draft",
           "load", "make_desc", "prefill_min_workspace_size", "prefill_path",
           "prefill_workspace_size", "read_device_status", "causal_conv", "causal_conv_backward",
           "causal_conv_decode", "causal_conv_draft", "commit_draft", "gated_decode",
           "gated_decode_draft", "gated_scan", "gated_scan_backward", "sample", "sample_probs", "ssm_decode",
           "ssm_decode_draft", "ssm_scan", "ssm_scan_workspace_size", "verify_draft"]
