"""Verification through the C boundary where operands may be missing."""
import ctypes

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import layer

pytestmark = pytest.mark.gpu


def test_no_tokens_at_all_and_no_noise():
    """With no token in the batch the probabilities, tokens and noise may be missing."""
    n = 3
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    kept, nxt = (torch.full((n,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    lib, st = layer._load(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rc = lib.kda_verify_draft(n, 0, 1000, None, None, None, None, None, cu.data_ptr(), kept.data_ptr(),
                              nxt.data_ptr(), ws.data_ptr(), 256, st)
    assert rc == 0 and kda.read_device_status(ws) == 0
    assert kept.tolist() == [0] * n and nxt.tolist() == [-1] * n
