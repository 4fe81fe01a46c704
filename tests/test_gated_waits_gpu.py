"""The bound of the gated recurrence's waits: tiles that wait for the tiles before them give up after it, which the
status says, in either pass; the next call starts clean and gives what it gave.  (The bound is a nanosecond: a single
sequence's later tiles wait for tens of microseconds, as many trips to the L2 as groups of tiles come before them.)"""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api
from tests.test_gated_gpu import BF, F32, _back, _clean, _inputs, _scan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,ch", [(BF, 64), (F32, 32)])
def test_a_bound_that_no_wait_keeps_is_reported(dtype, ch):
    lens = [20000]
    d = _inputs(lens, ch, dtype, seed=1)
    want = _scan(d, lens, output_carries=True)
    grads = _back(d, lens, want[2])
    torch.cuda.synchronize()
    api.set_pipeline_wait_limit(1)
    try:
        _scan(d, lens)
        assert kda.read_device_status(kda.gated_scan.last_workspace) == 4
        _back(d, lens, want[2])
        assert kda.read_device_status(kda.gated_scan_backward.last_workspace) == 4
    finally:
        api.set_pipeline_wait_limit(0)
    assert all(torch.equal(a, b) for a, b in zip(want, _scan(d, lens, output_carries=True)))
    _clean(kda.gated_scan)
    assert all(torch.equal(a, b) for a, b in zip(grads, _back(d, lens, want[2])))
    _clean(kda.gated_scan_backward)
