"""The tensor-core scan where steps are small, element by element."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from tests import _layer_ref as ref
from tests.test_ssm_decays_gpu import _inputs

pytestmark = pytest.mark.gpu
BF, F32 = ref.BF, ref.F32


def test_small_steps_keep_their_relative_accuracy():
    """From a zero state a token leaves S = d b x.  d = softplus(dt + dt_bias) is good to 4e-7 at any size
    (the exponential 2^-22, its exact argument, a quotient, the series); S's three parts add up with two
    more roundings of 2^-23 and the weighted x has one of 2^-24: 4e-7 + 3e-7."""
    H, K, V, n = 64, 64, 64, 6
    d, g = _inputs([1] * n, H, 1, K, V, seed=3)
    bias = torch.rand(H, generator=g) * -57 - 3
    bias[:8] = torch.tensor([0.0, -1.0, -3.0, -10.0, -20.0, -40.0, -50.0, -60.0])
    dt = (d["dt"] * 2).to(BF)
    c = lambda t: t.cuda()
    _, S = kda.ssm_scan(c(d["x"]), c(dt), c(torch.zeros(H)), c(d["B"]), c(d["C"]),
                        ref.cu_of([1] * n).cuda(), dt_bias=c(bias))
    z = (dt.float() + bias).double()  # the sum is made in fp32
    step = torch.logaddexp(z, torch.zeros_like(z))
    want = step[..., None, None] * d["B"].double()[:, :, :, None] * d["x"].double()[:, :, None, :]
    err = ((S.double().cpu() - want).abs() / want.abs())[want.abs() > 1e-30]
    assert float(err.max()) <= 7e-7, float(err.max())
