"""The draw of tokens without a GPU: refusals of the binding and of the C boundary, and the table of the
kernel's exponential."""
import ctypes
import os
import re
import subprocess
from fractions import Fraction

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import layer

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
N, V = 4, 100
FAKE = 1 << 20  # never dereferenced


@pytest.mark.parametrize("over,err", [
    (dict(logits=torch.zeros(N, V, dtype=torch.float16)), TypeError), (dict(logits=torch.zeros(V)), ValueError),
    (dict(logits=torch.zeros(N, 0)), ValueError), (dict(logits=torch.zeros(V, N).T), ValueError),
    (dict(logits=torch.zeros(1, V).expand(N, V)), ValueError),
    (dict(noise=torch.zeros(N, V, dtype=BF)), TypeError), (dict(noise=torch.zeros(N, V - 1)), ValueError),
    (dict(temperature=torch.ones(N, dtype=BF)), TypeError), (dict(temperature=torch.ones(N + 1)), ValueError),
    (dict(temperature=-1.0), ValueError), (dict(temperature=float("nan")), ValueError), (dict(temperature="1"), TypeError),
    (dict(top_k=torch.ones(N)), TypeError), (dict(top_k=1.5), TypeError), (dict(top_k=1 << 31), ValueError),
    (dict(top_k=True), TypeError),
    (dict(top_p=torch.ones(N, 1)), ValueError), (dict(top_p=float("nan")), ValueError),
    (dict(min_p=torch.ones(N, dtype=torch.float64)), TypeError), (dict(min_p=float("nan")), ValueError),
    (dict(out=torch.zeros(N)), TypeError), (dict(out=torch.zeros(N + 1, dtype=I32)), ValueError),
    (dict(), ValueError),                        # nothing wrong but the device
])
def test_binding_refuses(over, err):
    a = dict(dict(logits=torch.zeros(N, V), noise=torch.ones(N, V)), **over)
    with pytest.raises(err):
        kda.sample(a.pop("logits"), a.pop("noise"), **a)
    if "noise" not in over and "out" not in over:
        a = dict(dict(logits=torch.zeros(N, V)), **over)
        with pytest.raises(err):
            kda.sample_probs(a.pop("logits"), **a)


def _desc(**over):
    a = dict(num_rows=N, vocab=V, dtype=0, logits_pitch=V, noise_pitch=V, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    a.update(over)
    return layer.KdaSampleDesc(*a.values())


def test_c_boundary_refuses():
    lib, nan = layer._load(), float("nan")

    def sample(d=None, logits=FAKE, noise=FAKE, t=None, k=None, p=None, m=None, out=FAKE, ws=FAKE, nws=256):
        return lib.kda_sample(ctypes.byref(d or _desc()), logits, noise, t, k, p, m, out, ws, nws, None)

    def probs(d=None, logits=FAKE, t=None, k=None, p=None, m=None, out=FAKE, ws=FAKE, nws=256):
        return lib.kda_sample_probs(ctypes.byref(d or _desc()), logits, t, k, p, m, out, ws, nws, None)

    for call in (sample, probs):
        for over in (dict(num_rows=-1), dict(vocab=0), dict(dtype=2), dict(logits_pitch=V - 1), dict(temperature=-0.5),
                     dict(temperature=nan), dict(top_p=nan), dict(min_p=nan)):
            assert call(_desc(**over)) == 1, over
        for over in (dict(logits=None), dict(out=None), dict(ws=None), dict(ws=FAKE + 4), dict(logits=FAKE + 1),
                     dict(out=FAKE + 2), dict(t=FAKE + 2), dict(k=FAKE + 1), dict(p=FAKE + 2), dict(m=FAKE + 2)):
            assert call(**over) == 1, over
        assert call(nws=128) == 3
        assert call(_desc(vocab=360449, logits_pitch=360449, noise_pitch=360449)) == 2
        assert call(_desc(num_rows=(1 << 27) + 1)) == 2
    assert sample(noise=None) == 1 and sample(_desc(noise_pitch=V - 1)) == 1 and sample(noise=FAKE + 2) == 1


def test_descriptor_layout_matches_header(tmp_path):
    fields = [f for f, _ in layer.KdaSampleDesc._fields_]
    src = tmp_path / "layout.c"
    body = "\n".join(f'  printf("{f} %zu\\n", offsetof(kda_sample_desc_t, {f}));' for f in fields)
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kda.h"\nint main(void) {\n'
                   f'  printf("size %zu\\n", sizeof(kda_sample_desc_t));\n{body}\n  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include",
                    str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(layer.KdaSampleDesc)
    for f in fields:
        assert int(got[f]) == getattr(layer.KdaSampleDesc, f).offset, f


def test_table_of_powers():
    """Entry j is the whole number nearest to 2^(44 - j/32): (2 e - 1)^32 < 2^(32 * 45 - j) < (2 e + 1)^32."""
    src = open(os.path.join(ROOT, "linear_attention_prefill_chunked_gb300", "csrc", "kda_sample.cu")).read()
    table = [int(v) for v in re.findall(r"(\d+)ull", src[src.index("c_pow[32]"):src.index("struct Item")])]
    assert len(table) == 32 and table[0] == 1 << 44
    for j, e in enumerate(table[1:], 1):
        assert Fraction(2 * e - 1) ** 32 < Fraction(2) ** (32 * 45 - j) < Fraction(2 * e + 1) ** 32, j
