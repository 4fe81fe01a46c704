"""The gated recurrence, the convolution's backward pass and the draw of tokens as calls of the library: workspaces,
devices and streams, the bounds-checked build, other streams than the current one, two graphs of one workspace,
and the largest pitches."""
import os
import subprocess
import sys

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _calls():
    """Every entry point with small inputs, as functions of further arguments."""
    z = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device="cuda")
    cu = torch.tensor([0, 1, 3], dtype=I32, device="cuda")
    x, al, pool, w = z(3, 8), z(8), z(4, 8), z(8, 4)
    return dict(
        gated_scan=lambda **k: kda.gated_scan(x, x, al, cu, i=x, **k),
        gated_scan_backward=lambda **k: kda.gated_scan_backward(x, x, x, al, cu, z(1, 8), i=x, **k),
        gated_decode=lambda **k: kda.gated_decode(x, x, al, pool, i=x, **k),
        gated_decode_draft=lambda **k: kda.gated_decode_draft(x, x, al, cu, pool, i=x, max_steps=2, **k),
        causal_conv_backward=lambda **k: kda.causal_conv_backward(x, x, w, cu, **k),
        sample=lambda **k: kda.sample(x, x + 1, **k),
        sample_probs=lambda **k: kda.sample_probs(x, **k))


NAMES = ("gated_scan", "gated_scan_backward", "gated_decode", "gated_decode_draft", "causal_conv_backward", "sample",
         "sample_probs")


@pytest.mark.parametrize("name", NAMES)
def test_workspaces_and_devices(name, monkeypatch):
    call = _calls()[name]
    call()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    call(workspace=ws)
    assert getattr(kda, name).last_workspace is ws and kda.read_device_status(ws) == 0
    with pytest.raises(ValueError):
        call(workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        call(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(kda.KdaError):   # not on a boundary of 256 bytes
        call(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[8:])
    if name in ("gated_scan", "gated_scan_backward", "causal_conv_backward"):
        with pytest.raises(kda.KdaError):
            call(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name):
    """What an argument's stream has still to write is seen by a call on it, and its results by work behind it."""
    want = _calls()[name]()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)
        call = _calls()[name]
        got = call(stream=side)
    side.synchronize()
    flat = lambda o: [t for t in (o if isinstance(o, tuple) else (o,)) if t is not None]
    assert all(torch.equal(a, b) for a, b in zip(flat(want), flat(got)))


def test_two_graphs_of_one_workspace_replayed_in_turn():
    """A workspace holds nothing from one call to the next: graphs of other shapes that share one, replayed in any
    order on one stream, give what they gave."""
    g = torch.Generator().manual_seed(0)
    z = lambda *s: torch.randn(*s, generator=g).cuda()
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    graphs, outs, want, kept = [], [], [], []   # kept: a graph reads its inputs where they were
    for T, ch in ((700, 64), (90, 200)):
        x, r, i, al, dy = z(T, ch), z(T, ch), z(T, ch), z(ch), z(T, ch)
        w, logits = z(ch, 4), z(T, ch)
        cu = torch.tensor([0, T // 3, T], dtype=I32, device="cuda")

        def step(x=x, r=r, i=i, al=al, dy=dy, w=w, cu=cu, logits=logits):
            y, f, c = kda.gated_scan(x, r, al, cu, i=i, output_carries=True, workspace=ws)
            return (y, f, *kda.gated_scan_backward(dy, x, r, al, cu, c, i=i, workspace=ws)[:4],
                    *kda.causal_conv_backward(dy, x, w, cu, workspace=ws)[:2],
                    kda.sample_probs(logits, top_p=0.7, workspace=ws))

        kept.append(step)
        want.append([t.clone() for t in step()])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for k in (0, 1, 1, 0, 1, 0):
        for t in outs[k]:
            t.fill_(-1)
        graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[k], outs[k]))


def test_rows_more_than_32_bits_of_elements_apart():
    """Offsets past 2^31 elements: the last rows of a wide buffer."""
    pitch, T = (1 << 29) + 64, 9
    buf = torch.zeros(T * pitch, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(1)
    x, r, i, dy = (torch.randn(T, 64, generator=g).to(BF).cuda() for _ in range(4))
    wide = []
    for k, t in enumerate((x, r, i, dy)):
        v = buf.as_strided((T, 64), (pitch, 1), k * 64)
        v.copy_(t)
        wide.append(v)
    al, w = torch.zeros(64, device="cuda"), torch.randn(64, 4, generator=g).to(BF).cuda()
    cu = torch.tensor([0, 4, T], dtype=I32, device="cuda")
    a = kda.gated_scan(x, r, al, cu, i=i, output_carries=True)
    b = kda.gated_scan(wide[0], wide[1], al, cu, i=wide[2], output_carries=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a = kda.gated_scan_backward(dy, x, r, al, cu, a[2], i=i)
    b = kda.gated_scan_backward(wide[3], wide[0], wide[1], al, cu, b[2], i=wide[2])
    assert all(torch.equal(p, q) for p, q in zip(a[:4], b[:4]))
    a = kda.causal_conv_backward(dy, x, w, cu, activation="silu")
    b = kda.causal_conv_backward(wide[3], wide[0], w, cu, activation="silu")
    assert all(torch.equal(p, q) for p, q in zip(a[:2], b[:2]))
    noise = torch.rand(T, 64, generator=g).cuda() + 0.1
    assert torch.equal(kda.sample(x, noise, top_p=0.9), kda.sample(wide[0], noise, top_p=0.9))
    pool = torch.zeros(T, 64, device="cuda")
    other = pool.clone()
    assert torch.equal(kda.gated_decode(x, r, al, pool, i=i), kda.gated_decode(wide[0], wide[1], al, other, i=wide[2]))
    assert torch.equal(pool, other)


CHILD = r'''
import sys, torch
sys.path.insert(0, sys.argv[1])
import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api
from tests import test_gated_gpu as tg, test_conv_back_gpu as tb
assert api.debug_build() == (sys.argv[2] == "debug")
BF, F32 = torch.bfloat16, torch.float32
out = {}
def keep(name, fn, tensors):
    assert kda.read_device_status(fn.last_workspace) == 0, name
    out[name] = [t.cpu() for t in tensors if t is not None]
for dt, ch in ((BF, 264), (BF, 37), (F32, 70)):
    lens = [0, 5, 129, 1, 900]
    d = tg._inputs(lens, ch, dt)
    r = tg._scan(d, lens, output_carries=True)
    keep(f"gated {dt} {ch}", kda.gated_scan, r)
    keep(f"gated back {dt} {ch}", kda.gated_scan_backward, tg._back(d, lens, r[2]))
    pool = torch.ones(1040, ch, device="cuda")
    y = kda.gated_decode(d["x"], d["r"], d["A_log"], pool, i=d["i"])
    keep(f"gated token {dt} {ch}", kda.gated_decode, (y, pool))
    b = tb._inputs(lens, ch, 4, dt)
    keep(f"conv back {dt} {ch}", kda.causal_conv_backward, tb._back(b, lens, True))
g = torch.Generator().manual_seed(0)
for dt, vocab in ((F32, 20000), (BF, 3001)):
    z, noise = (torch.randn(6, vocab, generator=g) * 2).to(dt).cuda(), torch.rand(6, vocab, generator=g).cuda() + 0.01
    keep(f"sample {vocab}", kda.sample, (kda.sample(z, noise, top_k=100, top_p=0.9, min_p=0.01),))
    keep(f"probs {vocab}", kda.sample_probs, (kda.sample_probs(z, top_p=0.8), kda.sample_probs(z * 0, top_p=0.8)))
torch.save(out, sys.argv[3])
'''


def test_debug_build_clean_and_bit_identical(tmp_path):
    got = []
    for mode in ("release", "debug"):
        env = dict(os.environ)
        env.pop("KDA_DEBUG", None)
        if mode == "debug":
            env["KDA_DEBUG"] = "1"
        path = str(tmp_path / f"{mode}.pt")
        r = subprocess.run([sys.executable, "-c", CHILD, ROOT, mode, path], cwd=ROOT, env=env, capture_output=True,
                           text=True, timeout=900)
        assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
        got.append(torch.load(path))
    a, b = got
    assert sorted(a) == sorted(b)
    for name in a:
        for x, y in zip(a[name], b[name]):
            assert torch.equal(x, y), name
