"""Which device a call of the layer operators runs on: all tensors on one, a given workspace among them,
and that one current.  The checks themselves need no GPU (stand-ins of tensors); the calls do."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import layer


class On:
    """A tensor on a device, as far as the check looks."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.mark.parametrize("devices,current,fine", [
    ((0, 0, 0), 0, True), ((1, 1), 1, True), ((0, None, 0), 0, True),
    ((0, -1, 0), 0, False),      # one on the host
    ((0, 1), 0, False), ((0, 0, 1), 0, False), ((1, 0), 1, False),
    ((1, 1), 0, False),          # another than the current one
])
def test_one_device_and_the_current_one(devices, current, fine, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    args = [None if d is None else On(d) for d in devices]
    if fine:
        layer._cuda(*args)
    else:
        with pytest.raises(ValueError):
            layer._cuda(*args)


def test_streams_of_another_device_are_refused():
    class Stream:
        device_index, cuda_stream = 1, 77
    assert layer._stream(Stream, torch.device("cuda:1")) == 77
    with pytest.raises(ValueError):
        layer._stream(Stream, torch.device("cuda:0"))


def test_workspaces_must_be_contiguous():
    ws = torch.empty(512, dtype=torch.uint8)
    assert layer._workspace(None, ws, 256, ws.device) == (ws, 512)
    assert layer._workspace(None, ws[:100], 256, ws.device)[0].numel() == 256  # no room: a new one
    with pytest.raises(ValueError):
        layer._workspace(None, torch.empty(2048, dtype=torch.uint8)[::2], 256, ws.device)


def _calls():
    """Every entry point with small inputs, as functions of further arguments."""
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
    i32 = torch.int32
    cu = torch.tensor([0, 1, 3], dtype=i32, device="cuda")
    x, w, pool = z(3, 8), z(8, 4), z(4, 3, 8)
    xs, dt, a, b, states = z(3, 2, 64), z(3, 2), z(2), z(3, 1, 64), z(4, 2, 64, 64)
    return dict(
        causal_conv=lambda **k: kda.causal_conv(x, w, cu, **k),
        causal_conv_decode=lambda **k: kda.causal_conv_decode(x, w, pool, **k),
        causal_conv_draft=lambda **k: kda.causal_conv_draft(x, w, cu, pool, max_steps=2, **k),
        ssm_scan=lambda **k: kda.ssm_scan(xs, dt, a, b, b, cu, **k),
        ssm_decode=lambda **k: kda.ssm_decode(xs, dt, a, b, b, states, **k),
        ssm_decode_draft=lambda **k: kda.ssm_decode_draft(xs, dt, a, b, b, cu, states, max_steps=2, **k),
        verify_draft=lambda **k: kda.verify_draft(z(3, dt=i32), z(3, 5), z(3, 5), z(3), z(2, 5), cu, **k),
        commit_draft=lambda **k: kda.commit_draft(z(2, 2, 3, 8), z(2, dt=i32), pool, **k))


NAMES = ("causal_conv", "causal_conv_decode", "causal_conv_draft", "ssm_scan", "ssm_decode",
         "ssm_decode_draft", "verify_draft", "commit_draft")


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_calls_refuse_a_workspace_on_the_host_and_another_current_device(name, monkeypatch):
    call = _calls()[name]
    call()
    call(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        call(workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        call(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[::2])
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        call()
