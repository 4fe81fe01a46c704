"""The operators around the recurrence in the bounds-checked build (KDA_DEBUG=1): every status word
clean, results those of the normal build bit for bit."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys, torch
sys.path.insert(0, sys.argv[1])
import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api
from tests import _layer_ref as ref, test_conv_gpu as tc, test_ssm_gpu as ts, test_verify_gpu as tv
assert api.debug_build() == (sys.argv[2] == "debug")
BF, F32 = ref.BF, ref.F32
out = {}
def keep(name, fn, tensors):
    assert kda.read_device_status(fn.last_workspace) == 0, name
    out[name] = [t.cpu() for t in tensors]
for dt, ch, W in ((BF, 264, 4), (F32, 37, 3)):
    lens = [0, 5, 129, 1, 300]
    d = tc._inputs(lens, ch, W, dt)
    keep(f"conv {ch}", kda.causal_conv, kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), bias=d["b"],
                                                        activation="silu", state=d["h0"]))
    pool = torch.ones(440, W - 1, ch, device="cuda", dtype=dt)
    y = kda.causal_conv_decode(d["x"], d["w"], pool, bias=d["b"])
    keep(f"conv token {ch}", kda.causal_conv_decode, (y, pool))
for dt, core, lens in ((BF, False, [0, 5, 129, 2000]), (BF, True, [70, 3]), (F32, False, [1400, 1])):
    for K, V in ((128, 64), (64, 128)):
        d = ts._inputs(lens, 3, 1, K, V, dt)
        keep(f"scan {dt} {core} {K}", kda.ssm_scan, ts._scan(d, lens, state=d["h0"], cuda_core_path=core))
d = ts._inputs([1] * 9, 4, 2, 128, 64, BF)
pool = d["h0"].clone()
y = kda.ssm_decode(d["x"], d["dt"], d["A_log"], d["B"], d["C"], pool, D=d["D"], dt_bias=d["dt_bias"])
keep("scan token", kda.ssm_decode, (y, pool))
d = tv._inputs([3, 1, 4], 4001)
r = kda.verify_draft(d["tokens"], d["p"], d["q"], d["u"], d["noise"], ref.cu_of([3, 1, 4]).cuda())
keep("verify", kda.verify_draft, r)
cache = torch.arange(3 * 4 * 50, dtype=torch.float32, device="cuda").view(3, 4, 50)
pool = torch.zeros(5, 50, device="cuda")
kda.commit_draft(cache, r[0], pool)
keep("commit", kda.commit_draft, (pool,))
torch.save(out, sys.argv[3])
'''


def _child(mode, path):
    env = dict(os.environ)
    env.pop("KDA_DEBUG", None)
    if mode == "debug":
        env["KDA_DEBUG"] = "1"
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, mode, path], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


def test_debug_build_clean_and_bit_identical(tmp_path):
    import torch
    _child("release", str(tmp_path / "release.pt"))
    _child("debug", str(tmp_path / "debug.pt"))
    a, b = torch.load(tmp_path / "release.pt"), torch.load(tmp_path / "debug.pt")
    assert sorted(a) == sorted(b)
    for name in a:
        for x, y in zip(a[name], b[name]):
            assert torch.equal(x, y), name
