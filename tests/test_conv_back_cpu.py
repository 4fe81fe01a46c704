"""Refusals of the convolution's backward pass, by the binding and at the C boundary (no GPU)."""
import ctypes

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import layer

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
T, CH, W, N = 20, 48, 4, 3
FAKE = 1 << 20  # never dereferenced


@pytest.mark.parametrize("over,err", [
    (dict(dy=torch.zeros(T, CH)), TypeError), (dict(dy=torch.zeros(T, CH + 1, dtype=BF)), ValueError),
    (dict(dy=torch.zeros(1, CH, dtype=BF).expand(T, CH)), ValueError),
    (dict(dfinal=torch.zeros(N, W - 1, CH)), TypeError), (dict(dfinal=torch.zeros(N, W, CH, dtype=BF)), ValueError),
    (dict(state=torch.zeros(N + 1, W - 1, CH, dtype=BF)), ValueError), (dict(bias=torch.zeros(CH)), TypeError),
    (dict(), ValueError),                       # nothing wrong but the device
])
def test_binding_refuses(over, err):
    a = dict(dict(dy=torch.zeros(T, CH, dtype=BF)), **over)
    with pytest.raises(err):
        kda.causal_conv_backward(a.pop("dy"), torch.zeros(T, CH, dtype=BF), torch.zeros(CH, W, dtype=BF),
                                 torch.tensor([0, 5, 9, T], dtype=I32), **a)


def _call(lib, dtype=0, pitch=CH, dy=FAKE, dy_pitch=CH, x=FAKE, w=FAKE, b=FAKE, cu=FAKE, state=FAKE, dfinal=FAKE,
          dx=FAKE, dw=FAKE, db=FAKE, dstate=FAKE, ws=FAKE, nws=1 << 30, ch=CH, width=W):
    d = layer.KdaConvDesc(N, T, ch, width, dtype, 1, pitch, 0, 0)
    return lib.kda_causal_conv_backward(ctypes.byref(d), dy, dy_pitch, x, w, b, cu, state, dfinal, dx, dw, db, dstate,
                                        ws, nws, None)


def test_c_boundary_refuses():
    lib = layer._load()
    for over in (dict(dtype=2), dict(pitch=CH - 1), dict(dy_pitch=CH - 1), dict(width=5), dict(width=1), dict(ch=0),
                 dict(dy=None), dict(x=None), dict(w=None), dict(cu=None), dict(dx=None), dict(dw=None),
                 dict(ws=None), dict(ws=FAKE + 8), dict(dx=FAKE + 1), dict(state=FAKE + 1), dict(dfinal=FAKE + 1),
                 dict(dstate=FAKE + 1), dict(dw=FAKE + 2), dict(db=FAKE + 2)):
        assert _call(lib, **over) == 1, over
    assert _call(lib, nws=256) == 3
    big = 65535 * 32 + 1
    assert _call(lib, ch=big, pitch=big, dy_pitch=big) == 2
    size = lambda **k: lib.kda_causal_conv_backward_workspace_size(ctypes.byref(layer.KdaConvDesc(
        N, k.get("T", T), CH, k.get("W", W), 0, 1, CH, 0, 0)))
    least = 256 + 4 * (W + 1) * CH
    assert size() >= least + 4 * T and size(T=0) >= least and size(W=5) == 0
