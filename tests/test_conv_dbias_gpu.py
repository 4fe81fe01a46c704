"""The derivative by the bias at the C boundary, where it and the bias are pointers of their own: asked for without a
bias (which counts as zeros) it is that of a bias of zeros, not asked for with one nothing is written."""
import ctypes

import pytest
import torch

from linear_attention_prefill_chunked_gb300 import api, layer
from tests.test_conv_back_gpu import BF, F32, _inputs, _ref, cu_of

pytestmark = pytest.mark.gpu


def _call(d, lens, silu, bias, dbias):
    lib, (T, ch), W = layer._load(), d["x"].shape, d["w"].shape[1]
    dt = d["x"].dtype
    cu, dx = cu_of(lens).cuda(), torch.empty(T, ch, dtype=dt, device="cuda")
    dw, dstate = torch.empty(ch, W, device="cuda"), torch.empty(len(lens), W - 1, ch, dtype=dt, device="cuda")
    desc = layer.KdaConvDesc(len(lens), T, ch, W, api._dt(dt), int(silu), d["x"].stride(0), 0, 0)
    size = lib.kda_causal_conv_backward_workspace_size(ctypes.byref(desc))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    p = layer._p
    assert lib.kda_causal_conv_backward(
        ctypes.byref(desc), p(d["dy"]), d["dy"].stride(0), p(d["x"]), p(d["w"]), p(bias), p(cu), p(d["h0"]),
        p(d["dfinal"]), p(dx), p(dw), p(dbias), p(dstate), p(ws), size,
        torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    return dx, dw, dstate


@pytest.mark.parametrize("dtype,ch", [(BF, 64), (BF, 37), (F32, 36), (F32, 1)])
@pytest.mark.parametrize("silu", [True, False])
def test_bias_and_its_derivative_each_without_the_other(dtype, ch, silu):
    lens = [70, 0, 2, 300, 1]
    d = _inputs(lens, ch, 4, dtype, seed=ch)
    zero, guard = torch.zeros(ch, dtype=dtype, device="cuda"), torch.full((3, ch), 7.0, device="cuda")
    want = _call(d, lens, silu, zero, guard[0])
    got = _call(d, lens, silu, None, guard[1])
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(guard[0], guard[1])
    exact, err = _ref(dict(d, b=None), silu, lens)
    off = (guard[1].double().cpu() - exact["dbias"]).abs()
    assert (off <= 1.01 * err["dbias"] + 2.0 ** -24 * exact["dbias"].abs()).all()
    got = _call(d, lens, silu, zero, None)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and (guard[2] == 7.0).all()
