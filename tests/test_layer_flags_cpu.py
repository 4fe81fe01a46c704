"""Refusals at the C boundary and in the binding of the verification's flags and the commit's pool pitch
(no GPU)."""
import ctypes

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import layer


def test_unknown_verification_flags_are_refused():
    ok = ctypes.c_void_p(1 << 20)  # never dereferenced by these calls
    call = lambda flags, nws=256: layer._load().kda_verify_draft_marked(
        2, 5, 7, ok, ok, None, ok, ok, ok, ok, ok, flags, ok, nws, None)
    assert call(4) == 1 and call(0x80000001) == 1
    assert call(3, nws=8) == 3  # the flags pass: the workspace is what is refused


def test_commit_pool_pitches():
    cache, kept = torch.zeros(2, 3, 4, 8), torch.zeros(2, dtype=torch.int32)
    for pool, stride in ((torch.zeros(3, 40), 31), (torch.zeros(3, 40), -40), (torch.zeros(3, 30), 40),
                         (torch.zeros(0, 40), 40), (torch.zeros(3, 40), 0), (torch.zeros(120), 0)):
        with pytest.raises(ValueError, match="pool|cache"):
            kda.commit_draft(cache, kept, pool, slot_stride=stride)
    with pytest.raises(ValueError, match="CUDA"):  # fine but for the device
        kda.commit_draft(cache, kept, torch.zeros(3, 40), slot_stride=40)
