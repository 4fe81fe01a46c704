"""The short causal convolution against its definition in 64 bits: lengths from zero to several
tiles, odd channel counts, pitched rows, pool and dense states, drafts, invalid device data.

Bounds: a sum of W + 1 fp32 products and additions is off by at most (W + 2) 2^-24 of the sum of its
terms' magnitudes, and the result is rounded once to the output's type."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api
from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = ref.BF, ref.F32


def _inputs(lens, ch, W, dtype, seed=0, pitch=None, bias=True):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    wide = torch.randn(T, pitch or ch, generator=g).to(dtype)
    return dict(x=wide.cuda()[:, :ch], w=(torch.randn(ch, W, generator=g) * 0.5).to(dtype).cuda(),
                b=(torch.randn(ch, generator=g) * 0.1).to(dtype).cuda() if bias else None,
                h0=torch.randn(len(lens), W - 1, ch, generator=g).to(dtype).cuda())


def _check(y, want, x, w, dtype, what=""):
    """Element-wise: one rounding of the result, and the fp32 sum's own error."""
    y = y.double().cpu()
    assert torch.isfinite(y).all(), what
    size = float(w.double().abs().sum(1).max()) * float(x.double().abs().max()) + 1.0
    bound = ref.EPS[dtype] * 1.01 * want.abs() + size * (w.shape[1] + 6) * 2.0 ** -24 \
        + (2.0 ** -19 * want.abs() if dtype == BF else 0)  # the fast exponential of bf16 results
    assert ((y - want).abs() <= bound).all(), (what, float(((y - want).abs() - bound).max()))


LENS = [
    [1], [2, 1, 1, 3], [300], [0, 5, 0, 0, 129, 1, 0], [127, 1, 128, 3, 2, 2, 1, 17, 250],
    [15, 1, 16, 1, 1, 14, 2, 13, 3] * 5,
]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("ch,W,dtype", [(256, 4, BF), (264, 3, BF), (37, 4, BF), (1003, 3, F32),
                                        (64, 2, F32), (8, 2, BF), (1, 4, F32)])
def test_prompt_matches_definition(lens, ch, W, dtype):
    d = _inputs(lens, ch, W, dtype, seed=len(lens) + ch)
    for silu in (False, True):
        y, final = kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), bias=d["b"],
                                   activation="silu" if silu else None, state=d["h0"])
        want, fin, _ = ref.conv(d["x"], d["w"], d["b"], silu, lens, list(d["h0"]))
        assert kda.read_device_status(kda.causal_conv.last_workspace) == 0
        _check(y, want, d["x"], d["w"], dtype)
        assert torch.equal(final.double().cpu(), torch.stack(fin))  # copies of inputs: exact


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_state_no_bias_and_no_final(dtype):
    lens = [40, 3, 200]
    d = _inputs(lens, 96, 4, dtype, bias=False)
    y, final = kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), output_final_state=False)
    zero = [torch.zeros(3, 96)] * 3
    assert final is None
    _check(y, ref.conv(d["x"], d["w"], None, False, lens, zero)[0], d["x"], d["w"], dtype)


def test_pool_in_place_equals_dense_and_keeps_other_slots():
    lens = [3, 70, 0, 1, 130, 2, 16, 15]
    d = _inputs(lens, 136, 4, BF, seed=9)
    cu = ref.cu_of(lens).cuda()
    idx = torch.tensor([4, 0, 11, 2, -1, 7, 3, 9], dtype=torch.int32, device="cuda")
    pool = torch.randn(13, 3, 136, device="cuda").to(BF)
    slots = ref.slots_of(idx, 13)
    pool[slots] = d["h0"]
    before = pool.clone()
    yd, fd = kda.causal_conv(d["x"], d["w"], cu, bias=d["b"], activation="silu", state=d["h0"])
    yp, p = kda.causal_conv(d["x"], d["w"], cu, bias=d["b"], activation="silu", state=pool,
                            state_indices=idx)
    assert p is pool and torch.equal(yd, yp) and torch.equal(pool[slots], fd)
    rest = [i for i in range(13) if i not in slots]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("pitch", [256, 272, 257])  # packed, aligned and unaligned wider rows
def test_rows_of_a_wider_tensor(pitch):
    lens = [100, 33]
    d = _inputs(lens, 256, 4, BF, pitch=pitch)
    y, _ = kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), bias=d["b"], state=d["h0"])
    want, _, _ = ref.conv(d["x"], d["w"], d["b"], False, lens, list(d["h0"]))
    _check(y, want, d["x"], d["w"], BF)


def test_infinities_stay_in_their_sequence():
    lens = [20, 20, 20]
    d = _inputs(lens, 64, 4, BF)
    d["x"][20:40] = float("nan")
    d["h0"][1] = float("inf")
    y, final = kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), bias=d["b"], state=d["h0"])
    assert torch.isfinite(y[:20].float()).all() and torch.isfinite(y[40:].float()).all()
    assert torch.isfinite(final[0].float()).all() and torch.isfinite(final[2].float()).all()


def test_extreme_sums_of_silu():
    x = torch.tensor([[-300.0, 300.0, -20.0, 0.0, 80.0, -80.0, 1e-30, -1e-30]], device="cuda")
    w = torch.zeros(8, 2, device="cuda")
    w[:, 1] = 1.0
    for dtype in (F32, BF):
        y, _ = kda.causal_conv(x.to(dtype), w.to(dtype), ref.cu_of([1]).cuda(), activation="silu")
        want = torch.nn.functional.silu(x.to(dtype).double())
        assert torch.allclose(y.double(), want, rtol=2 * ref.EPS[dtype] + 2e-6, atol=1e-37)


@pytest.mark.parametrize("rows,ch,W,dtype", [(1, 8, 4, BF), (5, 12288, 4, BF), (33, 77, 3, F32),
                                             (7, 31, 2, BF)])
def test_token_matches_definition(rows, ch, W, dtype):
    d = _inputs([1] * rows, ch, W, dtype, seed=rows)
    pool = torch.randn(rows + 4, W - 1, ch, device="cuda").to(dtype)
    idx = torch.randperm(rows + 3)[:rows].to(torch.int32).cuda()
    idx[0] = -1
    slots = ref.slots_of(idx, rows + 4)
    before = pool.clone()
    y = kda.causal_conv_decode(d["x"], d["w"], pool, idx, bias=d["b"], activation="silu")
    want, fin, _ = ref.conv(d["x"], d["w"], d["b"], True, [1] * rows, list(before[slots]))
    _check(y, want, d["x"], d["w"], dtype)
    assert torch.equal(pool[slots].double().cpu(), torch.stack(fin))
    rest = [i for i in range(rows + 4) if i not in slots]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("update", [False, True])
@pytest.mark.parametrize("ch,dtype", [(128, BF), (45, F32)])
def test_draft_steps(update, ch, dtype):
    lens = [4, 1, 0, 3, 2]
    d = _inputs(lens, ch, 4, dtype, seed=2)
    pool = torch.randn(5, 3, ch, device="cuda").to(dtype)
    before = pool.clone()
    cache = torch.full((5, 6, 3, ch), 7.0, device="cuda", dtype=dtype)
    y = kda.causal_conv_draft(d["x"], d["w"], ref.cu_of(lens).cuda(), pool, bias=d["b"],
                              cache=cache, max_steps=4, update_state=update)
    want, fin, steps = ref.conv(d["x"], d["w"], d["b"], False, lens, list(before))
    _check(y, want, d["x"], d["w"], dtype)
    for n, each in enumerate(steps):
        for j, h in enumerate(each):
            assert torch.equal(cache[n, j].double().cpu(), h)
        assert (cache[n, len(each):] == 7).all()
    assert torch.equal(pool.double().cpu(), torch.stack(fin) if update else before.double().cpu())


def test_token_by_token_equals_prompt():
    lens = [50]
    d = _inputs(lens, 40, 4, F32)
    y, final = kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), bias=d["b"], state=d["h0"])
    pool = d["h0"].clone()
    each = [kda.causal_conv_decode(d["x"][t:t + 1], d["w"], pool, bias=d["b"]) for t in range(50)]
    assert torch.equal(torch.cat(each), y) and torch.equal(pool, final)


def test_bad_device_data_is_skipped_and_reported():
    lens = [10, 20, 30]
    d = _inputs(lens, 64, 4, BF)
    pool = torch.randn(6, 3, 64, device="cuda").to(BF)
    out = torch.full((60, 64), 7.0, device="cuda", dtype=BF)
    good = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    want, _ = kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), state=pool.clone(), state_indices=good)
    bad = torch.tensor([0, 6, 2], dtype=torch.int32, device="cuda")
    p = pool.clone()
    kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), state=p, state_indices=bad, out=out)
    assert kda.read_device_status(kda.causal_conv.last_workspace) == api.KDA_DEVICE_BAD_SLOT
    assert (out[10:30] == 7).all() and torch.equal(out[:10], want[:10]) and torch.equal(out[30:], want[30:])
    assert torch.equal(p[3:], pool[3:])
    cu = torch.tensor([0, 10, 5, 60], dtype=torch.int32, device="cuda")  # the middle one runs backwards
    kda.causal_conv(d["x"], d["w"], cu, state=pool.clone(), state_indices=good, out=out)
    assert kda.read_device_status(kda.causal_conv.last_workspace) == api.KDA_DEVICE_BAD_SEQLENS
    cu = torch.tensor([0, 10, 30, 61], dtype=torch.int32, device="cuda")  # past the last row
    out.fill_(7)
    kda.causal_conv(d["x"], d["w"], cu, state=pool.clone(), state_indices=good, out=out)
    assert kda.read_device_status(kda.causal_conv.last_workspace) == api.KDA_DEVICE_BAD_SEQLENS
    assert torch.equal(out[:30], want[:30]) and (out[30:] == 7).all()
    cache = torch.zeros(3, 10, 3, 64, device="cuda", dtype=BF)
    kda.causal_conv_draft(d["x"], d["w"], ref.cu_of(lens).cuda(), pool.clone(), good, cache=cache,
                          max_steps=10)
    assert kda.read_device_status(kda.causal_conv_draft.last_workspace) == api.KDA_DEVICE_BAD_SEQLENS


def test_another_stream_and_an_empty_batch():
    lens = [64, 64]
    d = _inputs(lens, 512, 4, BF)
    want, wf = kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), state=d["h0"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, f = kda.causal_conv(d["x"], d["w"], ref.cu_of(lens).cuda(), state=d["h0"], stream=s)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(f, wf)
    y, f = kda.causal_conv(d["x"][:0], d["w"], ref.cu_of([]).cuda())
    assert y.shape == (0, 512) and f.shape == (0, 3, 512)
    y, f = kda.causal_conv(d["x"][:0], d["w"], ref.cu_of([0, 0]).cuda(), state=d["h0"])
    assert torch.equal(f, d["h0"])
