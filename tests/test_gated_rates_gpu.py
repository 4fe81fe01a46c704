"""The gated recurrence under rates from slow to the largest that count, over states whose product with the
log-decay passes the largest fp32 number: where the decay is 0 so is all that a derivative takes of it.  Bounds as in
``_gated_ref``, which gets e^100 for an infinite rate (a decay of 0 as well), and 2^-100: a decay below 2^-126 counts
as 0, times a rate's exponent of 104 and states and derivatives below 2^10."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from tests import _gated_ref as ref
from tests.test_gated_gpu import BF, F32, _back, _clean, _inputs, _ref, _scan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,gate,pitch", [(BF, True, 0), (BF, False, 1), (F32, True, 0)])
@pytest.mark.parametrize("lens", [[1], [200], [90, 0, 40, 1, 7]])
def test_largest_rates(dtype, gate, pitch, lens):
    al = torch.tensor([-3.0, 0.0, 2.0, 3.0, 4.0, 5.0, 10.0, 40.0, 80.0, 87.0, 88.0, 88.5, 89.0, 100.0, float("inf"),
                       88.7])
    d = _inputs(lens, al.numel(), dtype, seed=5, gate=gate, pitch=pitch)
    d = dict(d, A_log=al.cuda(), x=d["x"] * 64, h0=d["h0"] * 64)
    y, final, carries = _scan(d, lens, output_carries=True)
    _clean(kda.gated_scan)
    k = _ref(dict(d, A_log=al.clamp(max=100.0)), lens)
    ref.check(y, k["y"], k["err"] + 2.0 ** -100, dtype, "y")
    want, err = ref.backward(k, d["dy"], d["dfinal"], lens)
    for name, t in zip(("dx", "dr", "di", "dA_log", "dstate"), _back(d, lens, carries)):
        if t is not None:
            ref.check(t, want[name], err[name] + 2.0 ** -100, dtype if name in ("dx", "dr", "di") else F32, name)
    _clean(kda.gated_scan_backward)


@pytest.mark.parametrize("dtype,ch_gate", [(BF, True), (BF, False), (F32, True)])
def test_shut_and_open_gates_under_the_largest_rates(dtype, ch_gate):
    """A shut gate keeps the state whole whatever the rate, and has no derivative; an open one leaves nothing of it.
    (r between -103 and -87, where sigmoid(r) is no normal number and counts as 0, is not among them.)"""
    lens = [70, 1, 40]
    rates = torch.tensor([0.0, 5.0, 60.0, 75.0, 80.0, 88.0, 100.0, float("inf")])
    al = rates.repeat(4)
    d = _inputs(lens, al.numel(), dtype, seed=6, gate=ch_gate)
    r = d["r"].clone()
    for j, v in enumerate((-250.0, -300.0, float("-inf"), float("inf"))):
        r[:, 8 * j:8 * j + 8] = v
        r[3::7, 8 * j:8 * j + 8] = 1.5     # some rows forget
    d = dict(d, r=r, A_log=al.cuda())
    y, final, carries = _scan(d, lens, output_carries=True)
    _clean(kda.gated_scan)
    k = _ref(dict(d, A_log=al.clamp(max=100.0)), lens)
    # a shut gate's sqrt(1 - a^2) is 0 here, and sqrt(2 e^(100 - 250)) < 2^-107 at most in the 64-bit form, times inputs
    # below 8, derivatives below 2^6 and 111 rows
    slack = 2.0 ** -90
    ref.check(y, k["y"], k["err"] + slack, dtype, "y")
    want, err = ref.backward(k, d["dy"], d["dfinal"], lens)
    for name, t in zip(("dx", "dr", "di", "dA_log", "dstate"), _back(d, lens, carries)):
        if t is not None:
            ref.check(t, want[name], err[name] + slack, dtype if name in ("dx", "dr", "di") else F32, name)
    _clean(kda.gated_scan_backward)
