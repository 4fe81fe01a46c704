"""Workspace sizes of the state space scan (no GPU): room for cuts only where a sequence can be cut."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import layer


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,G,K,V", [(64, 1, 128, 64), (32, 8, 128, 128), (3, 3, 64, 64)])
def test_room_for_cuts_is_asked_for_where_there_can_be_any(dtype, H, G, K, V):
    size = lambda n, t: kda.ssm_scan_workspace_size(layer.ssm_desc(n, t, H, G, K, V, dtype))
    state = H * K * V * 4
    for n in (1, 40):
        assert size(n, 0) == size(n, 1) == size(n, 1024) == layer.STATUS_WORKSPACE_BYTES
        assert size(n, 1025) > 2 * state  # two parts of a cut sequence at least
        assert size(n, 1025) == size(n, 1 << 20)
