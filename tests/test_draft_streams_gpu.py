"""Draft steps on a stream of their own: the most steps of a request, when not given, are read in that
stream's order."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda

pytestmark = pytest.mark.gpu


def _late(cu, value, stream):
    """Writes cu on the stream after some milliseconds of other work there."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
        cu.copy_(value)


def test_max_steps_is_read_after_the_streams_work():
    s = torch.cuda.Stream()
    lens = torch.tensor([0, 4, 5], dtype=torch.int32, device="cuda")
    x, w = torch.randn(5, 64, device="cuda"), torch.randn(64, 4, device="cuda")
    pool = torch.randn(3, 3, 64, device="cuda")
    want = kda.causal_conv_draft(x, w, lens, pool)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    _late(cu, lens, s)
    got = kda.causal_conv_draft(x, w, cu, pool, stream=s)
    s.synchronize()
    assert kda.read_device_status(kda.causal_conv_draft.last_workspace) == 0
    assert torch.equal(got, want)

    H, K, V = 2, 64, 64
    xs, dt = torch.randn(5, H, V, device="cuda"), torch.randn(5, H, device="cuda")
    B, C = torch.randn(5, 1, K, device="cuda"), torch.randn(5, 1, K, device="cuda")
    a, states = torch.zeros(H, device="cuda"), torch.randn(3, H, K, V, device="cuda")
    want = kda.ssm_decode_draft(xs, dt, a, B, C, lens, states)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    _late(cu, lens, s)
    got = kda.ssm_decode_draft(xs, dt, a, B, C, cu, states, stream=s)
    s.synchronize()
    assert kda.read_device_status(kda.ssm_decode_draft.last_workspace) == 0
    assert torch.equal(got, want)
