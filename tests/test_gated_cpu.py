"""The gated recurrence without a GPU: the reference's derivatives against differences of its own forward
pass, and the refusals of the binding and of the C boundary, before any launch."""
import ctypes
import os
import subprocess

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import layer
from tests import _gated_ref as ref

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, CH, N = 20, 48, 3


@pytest.mark.parametrize("gate", [True, False])
def test_reference_derivatives_against_differences(gate):
    g = torch.Generator().manual_seed(0)
    lens, ch = [4, 0, 5], 5
    z = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    args = [z(9, ch), z(9, ch), z(9, ch) if gate else None, z(ch), z(3, ch)]
    dy, dfinal = z(9, ch), z(3, ch)

    def run(x, r, i, al, h0):
        return ref.forward(x, r, i, al, lens, list(h0), F32)

    def loss(*a):
        k = run(*a)
        return float((k["y"] * dy).sum() + (k["final"] * dfinal).sum())

    want, _ = ref.backward(run(*args), dy, dfinal, lens)
    for at, name in enumerate(("dx", "dr", "di", "dA_log", "dstate")):
        if args[at] is None:
            continue
        v, step = z(*args[at].shape), 1e-5
        a, b = list(args), list(args)
        a[at], b[at] = args[at] + step * v, args[at] - step * v
        # a central difference's error: step^2 / 6 of a third derivative of a few units, and 2^-53 / step
        assert abs((loss(*a) - loss(*b)) / (2 * step) - float((want[name] * v).sum())) < 1e-8, name


def _args(**over):
    a = dict(x=torch.zeros(T, CH, dtype=BF), r=torch.zeros(T, CH, dtype=BF), A_log=torch.zeros(CH),
             i=torch.zeros(T, CH, dtype=BF), cu_seqlens=torch.tensor([0, 5, 9, T], dtype=I32),
             state=torch.zeros(N, CH))
    a.update(over)
    return layer.check_gated_args(a.pop("x"), a.pop("r"), a.pop("A_log"), **a)


def test_arguments():
    assert _args() == (N, T, CH, (CH, CH, CH))
    both = torch.zeros(T, 100, dtype=BF)
    assert _args(r=both[:, 1:49], i=both[:, 50:98])[-1] == (CH, 100, 100)
    assert _args(i=None)[-1] == (CH, CH, CH)
    _args(state=torch.zeros(9, CH), state_indices=torch.zeros(N, dtype=I32))
    _args(state=torch.zeros(9, 50), state_indices=torch.zeros(N, dtype=I32), slot_stride=50)


@pytest.mark.parametrize("over,err", [
    (dict(x=torch.zeros(T, CH)), TypeError),
    (dict(x=torch.zeros(T, CH, dtype=torch.float16)), TypeError),
    (dict(x=torch.zeros(T, CH, 1, dtype=BF)), ValueError),
    (dict(r=torch.zeros(T, CH)), TypeError),
    (dict(r=torch.zeros(T - 1, CH, dtype=BF)), ValueError),
    (dict(i=torch.zeros(CH, T, dtype=BF).T), ValueError),
    (dict(i=torch.zeros(1, CH, dtype=BF).expand(T, CH)), ValueError),
    (dict(A_log=torch.zeros(CH, dtype=BF)), TypeError),
    (dict(A_log=torch.zeros(CH + 1)), ValueError),
    (dict(cu_seqlens=torch.tensor([0, T])), TypeError),
    (dict(state=torch.zeros(N, CH, dtype=BF)), TypeError),
    (dict(state=torch.zeros(N + 1, CH)), ValueError),
    (dict(final_state=torch.zeros(N, CH, dtype=BF)), TypeError),
    (dict(state=None, state_indices=torch.zeros(N, dtype=I32)), ValueError),
    (dict(state=torch.zeros(9, CH, dtype=BF), state_indices=torch.zeros(N, dtype=I32)), TypeError),
    (dict(state=torch.zeros(9, 40), state_indices=torch.zeros(N, dtype=I32), slot_stride=40), ValueError),
    (dict(state=torch.zeros(9, CH), state_indices=torch.zeros(N, dtype=I32), final_state=torch.zeros(9, CH)),
     ValueError),
    (dict(out=torch.zeros(T, CH)), TypeError),
])
def test_refusals(over, err):
    with pytest.raises(err):
        _args(**over)


def test_backward_refusals():
    x, al = torch.zeros(T, CH), torch.zeros(CH)
    cu, c = torch.tensor([0, T], dtype=I32), torch.zeros(1, CH)
    for bad, err in ((dict(dy=torch.zeros(T, CH, dtype=BF)), TypeError), (dict(dy=torch.zeros(T, CH - 1)), ValueError),
                     (dict(carries=torch.zeros(2, CH)), ValueError),
                     (dict(carries=torch.zeros(1, CH, dtype=BF)), TypeError),
                     (dict(dfinal=torch.zeros(2, CH)), ValueError), (dict(state=torch.zeros(2, CH)), ValueError),
                     (dict(), ValueError)):  # nothing wrong but the device
        a = dict(dict(dy=x, carries=c), **bad)
        with pytest.raises(err):
            kda.gated_scan_backward(a.pop("dy"), x, x, al, cu, a.pop("carries"), **a)


def test_descriptor_layout_matches_header(tmp_path):
    fields = [f for f, _ in layer.KdaGatedDesc._fields_]
    src = tmp_path / "layout.c"
    body = "\n".join(f'  printf("{f} %zu\\n", offsetof(kda_gated_desc_t, {f}));' for f in fields)
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kda.h"\nint main(void) {\n'
                   f'  printf("size %zu\\n", sizeof(kda_gated_desc_t));\n{body}\n  return KDA_GATED_CARRY_ROWS - '
                   f"{layer.CARRY_ROWS};\n}}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include",
                    str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(layer.KdaGatedDesc)
    for f in fields:
        assert int(got[f]) == getattr(layer.KdaGatedDesc, f).offset, f


FAKE = 1 << 20  # never dereferenced: the calls below return first


def _desc(**over):
    a = dict(num_seqs=N, total_tokens=T, channels=CH, dtype=0, x_pitch=CH, r_pitch=CH, i_pitch=CH, num_slots=4,
             slot_stride_elems=0)
    a.update(over)
    return layer.KdaGatedDesc(*a.values())


BAD = [dict(num_seqs=-1), dict(total_tokens=-1), dict(total_tokens=1 << 31), dict(channels=0), dict(dtype=2),
       dict(x_pitch=CH - 1), dict(r_pitch=CH - 1), dict(i_pitch=CH - 1)]


def _scan(lib, d, x=FAKE, r=FAKE, i=FAKE, al=FAKE, cu=FAKE, state=FAKE, idx=FAKE, final=None, y=FAKE, carries=None,
          ws=FAKE, nws=1 << 30):
    return lib.kda_gated_scan(ctypes.byref(d), x, r, i, al, cu, state, idx, final, y, carries, ws, nws, None)


def _back(lib, d, dy=FAKE, pitch=CH, x=FAKE, r=FAKE, i=FAKE, al=FAKE, cu=FAKE, carries=FAKE, state=FAKE,
          dfinal=FAKE, dx=FAKE, dr=FAKE, di=FAKE, da=FAKE, dstate=FAKE, ws=FAKE, nws=1 << 30):
    return lib.kda_gated_scan_backward(ctypes.byref(d), dy, pitch, x, r, i, al, cu, carries, state, dfinal, dx, dr,
                                       di, da, dstate, ws, nws, None)


def _token(lib, d, x=FAKE, r=FAKE, i=FAKE, al=FAKE, cu=FAKE, pool=FAKE, idx=None, cache=None, pitch=0, steps=1,
           y=FAKE, ws=FAKE, nws=1 << 30):
    return lib.kda_gated_decode(ctypes.byref(d), x, r, i, al, cu, pool, idx, cache, pitch, steps, 1, y, ws, nws, None)


def test_c_boundary_refuses():
    lib = layer._load()
    for call in (_scan, _back, _token):
        for over in BAD:
            assert call(lib, _desc(**over)) == 1, (call, over)
        for null in ("x", "r", "al", "ws"):
            assert call(lib, _desc(), **{null: None}) == 1, (call, null)
        assert call(lib, _desc(), ws=FAKE + 16) == 1 and call(lib, _desc(), al=FAKE + 2) == 1
        assert call(lib, _desc(), x=FAKE + 1) == 1
        assert call(lib, _desc(), nws=128) == 3
    for over in (dict(cu=None), dict(y=None), dict(state=None), dict(final=FAKE + 256), dict(carries=FAKE + 2)):
        assert _scan(lib, _desc(), **over) == 1, over
    assert _scan(lib, _desc(num_slots=0)) == 1 and _scan(lib, _desc(slot_stride_elems=CH - 1)) == 1
    for over in (dict(dy=None), dict(pitch=CH - 1), dict(carries=None), dict(dx=None), dict(dr=None), dict(di=None),
                 dict(i=None), dict(da=None), dict(dstate=FAKE + 2), dict(dx=FAKE + 1)):
        assert _back(lib, _desc(), **over) == 1, over
    for over in (dict(cu=None), dict(pool=None), dict(steps=0), dict(cache=FAKE, pitch=CH - 1), dict(cache=FAKE + 2, pitch=CH)):
        assert _token(lib, _desc(), **over) == 1, over
    assert _token(lib, _desc(channels=1 << 30, x_pitch=1 << 30, r_pitch=1 << 30, i_pitch=1 << 30)) == 2
    big = _desc(total_tokens=(1 << 31) - 1, channels=1 << 12, x_pitch=1 << 12, r_pitch=1 << 12, i_pitch=1 << 12)
    assert _scan(lib, big, nws=1 << 62) == 2 and _back(lib, big, pitch=1 << 12, nws=1 << 62) == 2  # too many tiles
    assert lib.kda_gated_scan_workspace_size(ctypes.byref(big)) == 0
    assert lib.kda_gated_scan_workspace_size(ctypes.byref(_desc())) >= 256 + 4 * T
    assert lib.kda_gated_scan_backward_workspace_size(ctypes.byref(_desc(channels=0))) == 0
