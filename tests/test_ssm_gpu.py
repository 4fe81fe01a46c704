"""The selective state space scan against its recurrence in 64 bits.

Bounds (relative L2 over a tensor): fp32 results carry the rounding of fp32 sums of up to 128
products over a state with a memory of some hundred tokens, ~(128 + 100) 2^-24 at worst = 1.4e-5.
bf16 outputs are rounded once (2^-9 at most); in the tensor-core form the decayed scores and the
state that is read are bf16 operands too, each another 2^-9 at most of its part: 3 * 2^-9 in all.
States hold fp32 whatever the inputs' type, rounded once to a bf16 pool."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api
from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = ref.BF, ref.F32
Y_BOUND = {BF: 3 * 2.0 ** -9, F32: 2e-5}
S_BOUND = {BF: 2.0 ** -9 + 2e-5, F32: 2e-5}


def _inputs(lens, H, G, K, V, dtype, seed=0, sdt=F32, pitched=False, d=True, bias=True, a_max=16.0):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    n = lambda *s: torch.randn(*s, generator=g)
    step = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)
    out = dict(dt=n(T, H).to(dtype), A_log=torch.log(torch.rand(H, generator=g) * (a_max - 1) + 1),
               D=n(H) if d else None, dt_bias=torch.log(torch.expm1(step)) if bias else None,
               h0=(n(N, H, K, V) * 0.3).to(sdt))
    xbc = n(T, H * V + 2 * G * K).to(dtype).cuda()
    parts = xbc.split([H * V, G * K, G * K], 1)
    out = {k: (v.cuda() if v is not None else None) for k, v in out.items()}
    shapes = ((H, V), (G, K), (G, K))
    for name, p, s in zip(("x", "B", "C"), parts, shapes):
        out[name] = p.unflatten(1, s) if pitched else p.unflatten(1, s).contiguous()
    return out


def _scan(d, lens, **kw):
    a = dict(D=d["D"], dt_bias=d["dt_bias"])
    a.update(kw)
    return kda.ssm_scan(d["x"], d["dt"], d["A_log"], d["B"], d["C"], ref.cu_of(lens).cuda(), **a)


def _want(d, lens, h0):
    return ref.ssm(d["x"], d["dt"], d["A_log"], d["B"], d["C"], d["D"], d["dt_bias"], lens, h0)


def _close(y, fin, want, wfin, lens, dtype, sdt, what=""):
    assert ref.rel(y, want) <= Y_BOUND[dtype], (what, ref.rel(y, want))
    a = 0
    for i, n in enumerate(lens):  # every (sequence, head) on its own: a wrong one is off by ~1
        for h in range(y.shape[1]):
            if n:
                e = ref.rel(y[a:a + n, h], want[a:a + n, h])
                assert e <= 3 * Y_BOUND[dtype], (what, i, h, e)
            if fin is not None:
                e = ref.rel(fin[i, h], wfin[i][h])
                assert e <= 1.5 * S_BOUND[sdt], (what, "state", i, h, e)
        a += n


SHAPES = [(4, 2, 128, 128), (6, 1, 128, 64), (3, 3, 64, 64), (5, 1, 64, 128), (2, 2, 128, 64)]
LENS = [[1], [1, 2, 63, 64, 65], [0, 130, 0, 7, 200, 1], [513]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,G,K,V", SHAPES)
@pytest.mark.parametrize("dtype,cuda_core", [(BF, False), (BF, True), (F32, False)])
def test_prompt_matches_recurrence(lens, H, G, K, V, dtype, cuda_core):
    d = _inputs(lens, H, G, K, V, dtype, seed=H * 7 + len(lens), pitched=H % 2 == 0)
    y, fin = _scan(d, lens, state=d["h0"], cuda_core_path=cuda_core)
    assert kda.read_device_status(kda.ssm_scan.last_workspace) == 0
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    _close(y, fin, want, wfin, lens, dtype, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("with_d,with_bias", [(False, True), (True, False), (False, False)])
def test_optional_inputs_and_no_state(dtype, with_d, with_bias):
    lens = [100, 5]
    d = _inputs(lens, 4, 1, 128, 64, dtype, d=with_d, bias=with_bias, seed=3)
    y, fin = _scan(d, lens)
    want, wfin, _ = _want(d, lens, [torch.zeros(4, 128, 64)] * 2)
    _close(y, fin, want, wfin, lens, dtype, F32)
    y2, none = _scan(d, lens, output_final_state=False)
    assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sdt", [F32, BF])
def test_pool_in_place_equals_dense(dtype, sdt):
    lens = [70, 0, 3, 129]
    d = _inputs(lens, 4, 2, 128, 64, dtype, seed=5, sdt=sdt)
    idx = torch.tensor([3, 5, -1, 0], dtype=torch.int32, device="cuda")
    slots = ref.slots_of(idx, 8)
    pool = (torch.randn(8, 4, 128, 64, device="cuda") * 0.3).to(sdt)
    pool[slots] = d["h0"]
    before = pool.clone()
    yd, fd = _scan(d, lens, state=d["h0"])
    yp, p = _scan(d, lens, state=pool, state_indices=idx)
    assert p is pool and torch.equal(yd, yp) and torch.equal(pool[slots], fd)
    rest = [i for i in range(8) if i not in slots]
    assert torch.equal(pool[rest], before[rest])
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    _close(yd, fd, want, wfin, lens, dtype, sdt)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("a_max,shift", [(1000.0, 3.0), (1.001, -8.0)])
def test_strong_and_weak_decays(dtype, a_max, shift):
    """Log-decays from ~-1e4 a token (everything forgotten) to ~-1e-4 (nothing is)."""
    lens = [150, 64]
    d = _inputs(lens, 4, 1, 128, 64, dtype, seed=8, a_max=a_max)
    d["dt"] = (d["dt"].float() + shift).to(dtype)
    y, fin = _scan(d, lens, state=d["h0"])
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    _close(y, fin, want, wfin, lens, dtype, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_long_sequence_alone(dtype):
    """Few items and many chunks: the form that splits time."""
    lens = [2500]
    d = _inputs(lens, 2, 1, 128, 64, dtype, seed=11, a_max=2.0)
    y, fin = _scan(d, lens, state=d["h0"])
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    _close(y, fin, want, wfin, lens, dtype, F32)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")  # no room to split
    y2, fin2 = _scan(d, lens, state=d["h0"], workspace=small)
    _close(y2, fin2, want, wfin, lens, dtype, F32)
    y3, fin3 = _scan(d, lens, state=d["h0"])
    assert torch.equal(y, y3) and torch.equal(fin, fin3)


def test_many_sequences():
    lens = [(i * 37) % 90 for i in range(200)]
    d = _inputs(lens, 4, 1, 128, 64, BF, seed=12)
    y, fin = _scan(d, lens, state=d["h0"])
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    _close(y, fin, want, wfin, lens, BF, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_stay_in_their_sequence(dtype):
    lens = [20, 30, 20]
    d = _inputs(lens, 4, 1, 128, 64, dtype, seed=13)
    for name in ("x", "B", "C", "dt"):
        d[name][20:50] = float("nan")
    y, fin = _scan(d, lens, state=d["h0"])
    keep = [0, 2]
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    for a, i in ((0, 0), (50, 2)):
        assert ref.rel(y[a:a + 20], want[a:a + 20]) <= Y_BOUND[dtype]
        assert ref.rel(fin[i], wfin[i]) <= S_BOUND[F32], keep


@pytest.mark.parametrize("H,G,K,V", SHAPES)
@pytest.mark.parametrize("dtype,sdt", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
def test_token_matches_recurrence(H, G, K, V, dtype, sdt):
    rows = 9
    d = _inputs([1] * rows, H, G, K, V, dtype, seed=H, sdt=sdt, pitched=True)
    pool = (torch.randn(rows + 3, H, K, V, device="cuda") * 0.3).to(sdt)
    idx = torch.randperm(rows + 2)[:rows].to(torch.int32).cuda()
    idx[4] = -1
    slots = ref.slots_of(idx, rows + 3)
    before = pool.clone()
    y = kda.ssm_decode(d["x"], d["dt"], d["A_log"], d["B"], d["C"], pool, idx, D=d["D"],
                       dt_bias=d["dt_bias"])
    assert kda.read_device_status(kda.ssm_decode.last_workspace) == 0
    want, wfin, _ = _want(d, [1] * rows, list(before[slots]))
    _close(y, pool[slots], want, wfin, [1] * rows, dtype, sdt)
    rest = [i for i in range(rows + 3) if i not in slots]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("update", [False, True])
@pytest.mark.parametrize("K,V,sdt", [(128, 64, F32), (64, 128, BF)])
def test_draft_steps(update, K, V, sdt):
    lens = [4, 1, 0, 3]
    d = _inputs(lens, 4, 2, K, V, BF, seed=21, sdt=sdt)
    pool = d["h0"].clone()
    cache = torch.full((4, 5, 4, K, V), 7.0, device="cuda", dtype=sdt)
    y = kda.ssm_decode_draft(d["x"], d["dt"], d["A_log"], d["B"], d["C"], ref.cu_of(lens).cuda(), pool,
                             D=d["D"], dt_bias=d["dt_bias"], cache=cache, update_pool=update)
    want, wfin, steps = _want(d, lens, list(d["h0"]))
    assert ref.rel(y, want) <= Y_BOUND[BF]
    for n, each in enumerate(steps):
        for j, S in enumerate(each):
            assert ref.rel(cache[n, j], S) <= S_BOUND[sdt]
        assert (cache[n, len(each):] == 7).all()
    if update:
        for n in range(4):
            assert ref.rel(pool[n], wfin[n]) <= S_BOUND[sdt]
    else:
        assert torch.equal(pool, d["h0"])


def test_bad_device_data_is_skipped_and_reported():
    lens = [10, 20, 70]
    d = _inputs(lens, 4, 1, 128, 64, BF, seed=31)
    pool = torch.randn(5, 4, 128, 64, device="cuda") * 0.3
    good = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    bad = torch.tensor([0, -2, 2], dtype=torch.int32, device="cuda")
    for core in (False, True):
        want, wp = _scan(d, lens, state=pool.clone(), state_indices=good, cuda_core_path=core)
        out = torch.full_like(want, 7.0)
        p = pool.clone()
        _scan(d, lens, state=p, state_indices=bad, out=out, cuda_core_path=core)
        assert kda.read_device_status(kda.ssm_scan.last_workspace) == api.KDA_DEVICE_BAD_SLOT
        assert (out[10:30] == 7).all() and torch.equal(out[:10], want[:10])
        assert torch.equal(out[30:], want[30:]) and torch.equal(p[1], pool[1])
        assert torch.equal(p[2], wp[2])
        out.fill_(7)
        cu = torch.tensor([0, 10, 30, 101], dtype=torch.int32, device="cuda")
        kda.ssm_scan(d["x"], d["dt"], d["A_log"], d["B"], d["C"], cu, D=d["D"], dt_bias=d["dt_bias"],
                     state=pool.clone(), state_indices=good, out=out, cuda_core_path=core)
        assert kda.read_device_status(kda.ssm_scan.last_workspace) == api.KDA_DEVICE_BAD_SEQLENS
        assert (out[30:] == 7).all() and torch.equal(out[:30], want[:30])


def test_another_stream_and_an_empty_batch():
    lens = [64, 100]
    d = _inputs(lens, 4, 1, 128, 64, BF)
    want, wf = _scan(d, lens, state=d["h0"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, f = _scan(d, lens, state=d["h0"], stream=s)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(f, wf)
    e = {k: (v[:0] if k in ("x", "dt", "B", "C") else v) for k, v in d.items()}
    y, f = _scan(e, [])
    assert y.shape == (0, 4, 64) and f.shape == (0, 4, 128, 64)
    y, f = _scan(e, [0, 0], state=d["h0"])
    assert torch.equal(f, d["h0"])
