"""The short convolution with lengths that run backwards, so that sequences overlap: nothing outside the
tensor is read and what is good of the batch keeps its result."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,ch", [(BF, 64), (F32, 37)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("pool", [False, True])
def test_overlapping_sequences_read_nothing_outside(dtype, ch, W, pool):
    """[1, 12) and [0, 2) overlap, found by different warps of a block: whichever of them a token is
    given to, no input before the first row is read (there it would be NaN)."""
    cu = [1] + [12] * 39 + [0, 2]
    N = len(cu) - 1
    wide = torch.full((20, ch), float("nan"), device="cuda", dtype=dtype)
    wide[2:18] = torch.randn(16, ch, device="cuda").to(dtype)
    x = wide[2:18]
    w = torch.randn(ch, W, device="cuda").to(dtype)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for _ in range(20):
        state = torch.randn(N + 1, W - 1, ch, device="cuda").to(dtype)
        out = torch.zeros(16, ch, device="cuda", dtype=dtype)
        idx = torch.arange(N, dtype=torch.int32, device="cuda") if pool else None
        _, final = kda.causal_conv(x, w, cu, state=state if pool else state[:N], state_indices=idx,
                                   final_state=state if pool else state[:N].clone(), out=out)
        assert kda.read_device_status(kda.causal_conv.last_workspace) == api.KDA_DEVICE_BAD_SEQLENS
        assert torch.isfinite(out.float()).all() and torch.isfinite(final.float()).all()
        assert not out[12:].any()  # rows of no sequence


def test_sequences_before_the_bad_lengths_keep_their_results():
    lens, ch = [40, 3, 90], 128
    x = torch.randn(150, ch, device="cuda").to(BF)
    w = torch.randn(ch, 4, device="cuda").to(BF)
    good = torch.tensor([0, 40, 43, 133], dtype=torch.int32, device="cuda")
    want, _ = kda.causal_conv(x, w, good)
    bad = torch.tensor([0, 40, 43, 133, 130, 150], dtype=torch.int32, device="cuda")
    got, _ = kda.causal_conv(x, w, bad)
    assert kda.read_device_status(kda.causal_conv.last_workspace) == api.KDA_DEVICE_BAD_SEQLENS
    assert torch.equal(got[:130], want[:130])
    assert sum(lens) == 133
