"""Refusals of the operators around the recurrence, before any launch: the binding's checks of
shapes, types and strides, and the C boundary's of pointers, sizes and alignment (no GPU)."""
import ctypes
import os
import subprocess

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import layer

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, CH, W, N = 20, 48, 4, 3
H, G, K, V = 4, 2, 128, 64


def _conv(**over):
    a = dict(x=torch.zeros(T, CH, dtype=BF), weight=torch.zeros(CH, W, dtype=BF),
             bias=torch.zeros(CH, dtype=BF), cu_seqlens=torch.tensor([0, 5, 9, T], dtype=I32),
             state=torch.zeros(N, W - 1, CH, dtype=BF))
    a.update(over)
    x, w = a.pop("x"), a.pop("weight")
    return layer.check_conv_args(x, w, **a)


def test_conv_arguments():
    assert _conv() == (N, T, CH, W, CH)
    assert _conv(x=torch.zeros(T, 100, dtype=BF)[:, 3:51])[-1] == 100  # a slice of wider rows
    pool = torch.zeros(9, W - 1, CH, dtype=BF)
    _conv(state=pool, state_indices=torch.zeros(N, dtype=I32))
    _conv(state=torch.zeros(9, 200, dtype=BF), state_indices=torch.zeros(N, dtype=I32), slot_stride=200)


@pytest.mark.parametrize("over,err", [
    (dict(x=torch.zeros(T, CH)), TypeError),                              # weight of another type
    (dict(x=torch.zeros(T, CH, dtype=torch.float16)), TypeError),
    (dict(x=torch.zeros(CH, T, dtype=BF).T), ValueError),                 # columns, not rows, packed
    (dict(x=torch.zeros(1, CH, dtype=BF).expand(T, CH)), ValueError),     # rows that overlap
    (dict(weight=torch.zeros(CH, 5, dtype=BF)), ValueError),
    (dict(weight=torch.zeros(CH, 1, dtype=BF)), ValueError),
    (dict(weight=torch.zeros(CH + 1, W, dtype=BF)), ValueError),
    (dict(weight=torch.zeros(W, CH, dtype=BF).T), ValueError),
    (dict(bias=torch.zeros(CH - 1, dtype=BF)), ValueError),
    (dict(bias=torch.zeros(CH)), TypeError),
    (dict(cu_seqlens=torch.tensor([0, T])), TypeError),                   # int64
    (dict(state=torch.zeros(N, W, CH, dtype=BF)), ValueError),
    (dict(state=torch.zeros(N, W - 1, CH)), TypeError),
    (dict(final_state=torch.zeros(N - 1, W - 1, CH, dtype=BF)), ValueError),
    (dict(state=None, state_indices=torch.zeros(N, dtype=I32)), ValueError),
    (dict(state_indices=torch.zeros(N + 1, dtype=I32)), ValueError),
    (dict(state=torch.zeros(9, 100, dtype=BF), state_indices=torch.zeros(N, dtype=I32),
          slot_stride=100), ValueError),                                  # a pitch below a state
    (dict(out=torch.zeros(T, CH)), TypeError),
    (dict(out=torch.zeros(T - 1, CH, dtype=BF)), ValueError),
])
def test_conv_refusals(over, err):
    with pytest.raises(err):
        _conv(**over)


def _ssm(**over):
    a = dict(x=torch.zeros(T, H, V, dtype=BF), dt=torch.zeros(T, H, dtype=BF), A_log=torch.zeros(H),
             B=torch.zeros(T, G, K, dtype=BF), C=torch.zeros(T, G, K, dtype=BF), D=torch.zeros(H),
             dt_bias=torch.zeros(H), cu_seqlens=torch.tensor([0, 5, 9, T], dtype=I32),
             state=torch.zeros(N, H, K, V))
    a.update(over)
    pos = [a.pop(k) for k in ("x", "dt", "A_log", "B", "C")]
    return layer.check_ssm_args(*pos, **a)


def test_ssm_arguments():
    assert _ssm()[:6] == (N, T, H, G, K, V)
    wide = torch.zeros(T, H * V + 2 * G * K, dtype=BF)
    got = _ssm(x=wide[:, :H * V].unflatten(1, (H, V)), B=wide[:, H * V:H * V + G * K].unflatten(1, (G, K)))
    assert got[-1] == (768, H, 768, G * K)


@pytest.mark.parametrize("over,err", [
    (dict(x=torch.zeros(T, H, V)), TypeError),
    (dict(x=torch.zeros(T, H, 2 * V, dtype=BF)[:, :, ::2]), ValueError),
    (dict(x=torch.zeros(H, T, V, dtype=BF).transpose(0, 1)), ValueError),   # heads outermost
    (dict(x=torch.zeros(T, 3, V, dtype=BF)), ValueError),                   # not a multiple of G
    (dict(dt=torch.zeros(T - 1, H, dtype=BF)), ValueError),
    (dict(dt=torch.zeros(T, H)), TypeError),
    (dict(C=torch.zeros(T, G, 64, dtype=BF)), ValueError),
    (dict(A_log=torch.zeros(H, dtype=BF)), TypeError),
    (dict(A_log=None), TypeError),
    (dict(D=torch.zeros(H - 1)), ValueError),
    (dict(state=torch.zeros(N, H, V, K)), ValueError),
    (dict(final_state=torch.zeros(N, H, K, V, dtype=BF)), TypeError),
    (dict(state=None, token=True), ValueError),
    (dict(out=torch.zeros(T, H, V)), TypeError),
])
def test_ssm_refusals(over, err):
    with pytest.raises(err):
        _ssm(**over)


def test_verify_and_commit_refusals():
    vocab = 10
    ok = dict(tokens=torch.zeros(T, dtype=I32), target_probs=torch.zeros(T, vocab),
              draft_probs=torch.zeros(T, vocab), accept_u=torch.zeros(T), noise=torch.zeros(N, vocab),
              cu_seqlens=torch.tensor([0, 5, 9, T], dtype=I32))
    for over, err in ((dict(tokens=torch.zeros(T, dtype=torch.int64)), TypeError),
                      (dict(target_probs=torch.zeros(T, vocab, dtype=BF)), TypeError),
                      (dict(draft_probs=torch.zeros(T, vocab + 1)), ValueError),
                      (dict(accept_u=torch.zeros(T - 1)), ValueError),
                      (dict(noise=torch.zeros(N + 1, vocab)), ValueError),
                      (dict(target_probs=torch.zeros(vocab, T).T), ValueError),
                      ({}, ValueError)):                                    # not on a CUDA device
        with pytest.raises(err):
            kda.verify_draft(*dict(ok, **over).values())
    cache, kept, pool = torch.zeros(N, 4, 3, 8), torch.zeros(N, dtype=I32), torch.zeros(6, 3, 8)
    for c, k, p, err in ((cache.to(BF), kept, pool, TypeError), (cache, kept.long(), pool, TypeError),
                         (cache[:, :, :2], kept, pool, ValueError), (cache[:2], kept, pool, ValueError),
                         (cache.transpose(0, 1), kept, pool, ValueError),
                         (cache, kept, pool[:0], ValueError), (cache, kept, pool, ValueError)):
        with pytest.raises(err):
            kda.commit_draft(c, k, p)
    with pytest.raises(ValueError):
        layer._step_cache(torch.zeros(2, 3, 8), "cache", 2, 4, 8, F32)      # too few steps
    with pytest.raises(ValueError):
        layer._activation("gelu")


@pytest.mark.parametrize("cls,name", [(layer.KdaConvDesc, "kda_conv_desc_t"),
                                      (layer.KdaSsmInputs, "kda_ssm_inputs_t")])
def test_struct_layouts_match_header(cls, name, tmp_path):
    fields = [f for f, _ in cls._fields_]
    body = "\n".join(f'printf("{f} %zu\\n", offsetof({name}, {f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kda.h"\nint main(void) {\n'
                   f'printf("size %zu\\n", sizeof({name}));\n{body}\nreturn 0; }}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-I",
                    "/usr/local/cuda/include", str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(cls)
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f


def test_c_boundary_errors_return_before_any_launch():
    lib = layer._load()
    P, ref = ctypes.c_void_p, ctypes.byref
    ok, odd = P(1 << 20), P((1 << 20) + 2)  # never dereferenced by these calls

    def conv(ws=ok, nws=256, x=ok, cu=ok, state=None, idx=None, **kw):
        d = dict(num_seqs=3, total_tokens=20, channels=48, width=4, dtype=0, silu=0, x_pitch=48,
                 num_slots=0, slot_stride_elems=0)
        d.update(kw)
        return lib.kda_causal_conv(ref(layer.KdaConvDesc(*d.values())), x, ok, None, cu, state, idx,
                                   None, ok, ws, nws, None)

    for kw in (dict(width=5), dict(width=1), dict(channels=0), dict(dtype=7), dict(silu=2),
               dict(x_pitch=47), dict(num_seqs=-1), dict(x=None), dict(cu=None), dict(ws=None),
               dict(ws=P((1 << 20) + 64)), dict(idx=ok), dict(idx=ok, state=ok),
               dict(idx=ok, state=ok, num_slots=4, slot_stride_elems=100), dict(x=P((1 << 20) + 1))):
        assert conv(**kw) == 1, kw
    assert conv(nws=16) == 3 and conv(channels=1 << 30, x_pitch=1 << 30) == 2

    def ssm(nws=256, ws=ok, y=ok, state=None, idx=None, cu=ok, ins=None, **kw):
        d = layer.ssm_desc(3, 20, 4, 2, 128, 64, BF)
        for k, v in kw.items():
            setattr(d, k, v)
        i = dict(x=1 << 20, x_pitch=256, dt=1 << 20, dt_pitch=4, b=1 << 20, b_pitch=256, c=1 << 20,
                 c_pitch=256, a_log=1 << 20, dt_bias=None, d=None)
        i.update(ins or {})
        return lib.kda_ssm_scan(ref(d), ref(layer.KdaSsmInputs(*i.values())), cu, state, idx, None, y,
                                ws, nws, None)

    for kw in (dict(num_k_heads=3), dict(flags=2), dict(cu=None), dict(y=None), dict(y=odd),
               dict(ws=None), dict(idx=ok), dict(state=odd), dict(ins=dict(x=None)),
               dict(ins=dict(x_pitch=255)), dict(ins=dict(x_pitch=260)), dict(ins=dict(b=(1 << 20) + 2)),
               dict(ins=dict(dt_pitch=3)), dict(ins=dict(a_log=None)),
               dict(idx=ok, state=ok, num_slots=4, slot_stride_elems=4 * 128 * 64 + 4)):
        assert ssm(**kw) == 1, kw
    assert ssm(head_k_dim=96) == 2 and ssm(nws=0) == 3
    d = layer.ssm_desc(3, 20, 4, 2, 96, 64, BF)
    assert lib.kda_ssm_scan_workspace_size(ref(d)) == 0
    assert kda.ssm_scan_workspace_size(layer.ssm_desc(3, 20, 4, 2, 128, 64, BF)) >= 256
    one = layer.ssm_desc(3, 20, 4, 2, 128, 64, BF, num_slots=4)  # T must be N without cu_seqlens
    ins = layer.KdaSsmInputs(1 << 20, 256, 1 << 20, 4, 1 << 20, 256, 1 << 20, 256, 1 << 20, None, None)
    assert lib.kda_ssm_decode(ref(one), ref(ins), None, ok, None, None, 0, 1, 1, ok, ok, 256, None) == 1
    assert lib.kda_ssm_decode(ref(one), ref(ins), ok, ok, None, ok, 64, 1, 1, ok, ok, 256, None) == 1
    assert lib.kda_ssm_decode(ref(one), ref(ins), ok, ok, None, None, 0, 0, 1, ok, ok, 256, None) == 1
    v = lambda n=2, T=5, vocab=7, tok=ok, cu=ok, nws=256: lib.kda_verify_draft(
        n, T, vocab, tok, ok, None, ok, ok, cu, ok, ok, ok, nws, None)
    assert v(n=-1) == 1 and v(vocab=0) == 1 and v(tok=None) == 1 and v(cu=None) == 1
    assert v(nws=8) == 3 and v(tok=odd) == 1
    c = lambda n=2, dt=0, row=8, cache=ok, pitch=32, steps=4, pool=ok, slots=3, nws=256: \
        lib.kda_commit_draft(n, dt, row, cache, pitch, steps, ok, pool, slots, 0, None, ok, nws, None)
    assert c(dt=5) == 1 and c(row=0) == 1 and c(pitch=31) == 1 and c(steps=0) == 1 and c(slots=0) == 1
    assert c(cache=None) == 1 and c(dt=1, pool=odd) == 1 and c(nws=1) == 3
