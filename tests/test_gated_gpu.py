"""The gated linear recurrence against its definition in 64 bits: lengths from zero to many tiles, odd
channel counts, pitched rows, pool and dense states, the backward pass, tokens and drafts, invalid device
data, values that are no numbers, graphs and streams.  The bounds are those of ``_gated_ref``."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from tests import _gated_ref as ref
from tests._layer_ref import cu_of, slots_of

pytestmark = pytest.mark.gpu
BF, F32 = ref.BF, ref.F32


def _inputs(lens, ch, dtype, seed=0, gate=True, pitch=0):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    z = lambda *s: torch.randn(*s, generator=g)
    wide = z(T, 2 * ch + pitch).clamp(-8, 8).to(dtype).cuda()
    rate = -8.0 * torch.log(0.9 + 0.099 * torch.rand(ch, generator=g))
    return dict(x=z(T, ch).to(dtype).cuda(), r=wide[:, pitch:pitch + ch],
                i=wide[:, pitch + ch:] if gate else None, A_log=torch.log(rate).cuda(),
                dy=z(T, ch + pitch).to(dtype).cuda()[:, :ch], h0=z(N, ch).cuda(), dfinal=z(N, ch).cuda())


def _ref(d, lens, states=None):
    states = d["h0"] if states is None else states
    return ref.forward(d["x"], d["r"], d["i"], d["A_log"], lens, list(states))


def _scan(d, lens, **kw):
    kw.setdefault("state", d["h0"])
    return kda.gated_scan(d["x"], d["r"], d["A_log"], cu_of(lens).cuda(), i=d["i"], **kw)


def _back(d, lens, carries, **kw):
    kw.setdefault("state", d["h0"])
    kw.setdefault("dfinal", d["dfinal"])
    return kda.gated_scan_backward(d["dy"], d["x"], d["r"], d["A_log"], cu_of(lens).cuda(), carries, i=d["i"], **kw)


def _clean(fn):
    assert kda.read_device_status(fn.last_workspace) == 0


LENS = [[1], [2, 1, 1, 3], [127, 1, 128, 3, 2, 64, 1, 17, 250], [0, 5, 0, 0, 129, 1, 0], [700], [1] * 70]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("ch,dtype,gate,pitch", [(64, BF, True, 0), (70, BF, False, 2), (37, BF, True, 3),
                                                 (66, F32, True, 0), (1, F32, True, 1), (130, F32, False, 0)])
def test_prompt_and_backward_match_the_definition(lens, ch, dtype, gate, pitch):
    d = _inputs(lens, ch, dtype, seed=len(lens) + ch, gate=gate, pitch=pitch)
    y, final, carries = _scan(d, lens, output_carries=True)
    _clean(kda.gated_scan)
    k = _ref(d, lens)
    ref.check(y, k["y"], k["err"], dtype, "y")
    ends, at = [], 0
    for n in lens:
        at += n
        ends.append(at - 1 if n else None)
    bound = torch.stack([k["err"][e] if e is not None else torch.zeros(ch, dtype=torch.float64) for e in ends])
    ref.check(final, k["final"], bound, F32, "final")
    got = _back(d, lens, carries)
    _clean(kda.gated_scan_backward)
    want, err = ref.backward(k, d["dy"], d["dfinal"], lens)
    for name, t in zip(("dx", "dr", "di", "dA_log", "dstate"), got):
        if name == "di" and not gate:
            assert t is None
            continue
        ref.check(t, want[name], err[name], dtype if name in ("dx", "dr", "di") else F32, name)


@pytest.mark.parametrize("lens", [[5000], [2047, 1, 2049], [40, 3000, 0, 7, 2100]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequences_over_many_groups_of_tiles(lens, dtype):
    d = _inputs(lens, 44, dtype, seed=7)
    y, final, carries = _scan(d, lens, output_carries=True)
    k = _ref(d, lens)
    ref.check(y, k["y"], k["err"], dtype, "y")
    want, err = ref.backward(k, d["dy"], d["dfinal"], lens)
    for name, t in zip(("dx", "dr", "di", "dA_log", "dstate"), _back(d, lens, carries)):
        ref.check(t, want[name], err[name], dtype if name in ("dx", "dr", "di") else F32, name)
    _clean(kda.gated_scan)
    _clean(kda.gated_scan_backward)


def test_without_states():
    lens = [70, 0, 200]
    d = _inputs(lens, 40, BF, seed=3)
    y, final, carries = _scan(d, lens, state=None, output_carries=True)
    zero = torch.zeros(3, 40)
    k = _ref(d, lens, zero)
    ref.check(y, k["y"], k["err"], BF)
    assert torch.equal(final[1].cpu(), zero[1])
    y2, none = _scan(d, lens, state=None, output_final_state=False)
    assert none is None and torch.equal(y, y2)
    got = _back(d, lens, carries, state=None, dfinal=None)
    assert got[4] is None
    want, err = ref.backward(k, d["dy"], None, lens)
    for name, t in zip(("dx", "dr", "di", "dA_log"), got):
        ref.check(t, want[name], err[name], F32 if name == "dA_log" else BF, name)


def test_pool_in_place_equals_dense_and_keeps_other_slots():
    lens = [3, 70, 0, 1, 300, 2, 16, 15]
    for stride in (0, 140):
        d = _inputs(lens, 136, BF, seed=9)
        idx = torch.tensor([4, 0, 11, 2, -1, 7, 3, 9], dtype=torch.int32, device="cuda")
        buf = torch.randn(13, stride or 136, device="cuda")
        pool = buf if stride else buf.clone()
        slots = slots_of(idx, 13)
        pool[slots, :136] = d["h0"]
        before = pool.clone()
        yd, fd = _scan(d, lens)
        yp, p = _scan(d, lens, state=pool, state_indices=idx, slot_stride=stride)
        assert p is pool and torch.equal(yd, yp) and torch.equal(pool[slots, :136], fd)
        rest = [i for i in range(13) if i not in slots]
        assert torch.equal(pool[rest], before[rest]) and torch.equal(pool[:, 136:], before[:, 136:])


def test_in_place_dense_state():
    lens = [5, 0, 200]
    d = _inputs(lens, 64, F32, seed=2)
    y, f = _scan(d, lens)
    h = d["h0"].clone()
    y2, f2 = _scan(d, lens, state=h, final_state=h)
    assert f2 is h and torch.equal(f, h) and torch.equal(y, y2)


@pytest.mark.parametrize("dtype,ch", [(BF, 64), (BF, 37), (F32, 130)])
def test_tokens_and_drafts_follow_the_definition(dtype, ch):
    lens = [3, 1, 0, 4, 2]
    d = _inputs(lens, ch, dtype, seed=5)
    idx = torch.tensor([2, -1, 0, 5, 3], dtype=torch.int32, device="cuda")
    pool = torch.randn(8, ch, device="cuda")
    start = pool[slots_of(idx, 8)].clone()
    k = _ref(d, lens, start)
    cu, before = cu_of(lens).cuda(), pool.clone()
    cache = torch.full((5, 4, ch), -7.0, device="cuda")
    y = kda.gated_decode_draft(d["x"], d["r"], d["A_log"], cu, pool, idx, i=d["i"], cache=cache)
    _clean(kda.gated_decode_draft)
    ref.check(y, k["y"], k["err"], dtype)
    assert torch.equal(pool, before)
    at = 0
    for n, m in enumerate(lens):
        ref.check(cache[n, :m], k["y"][at:at + m], k["err"][at:at + m], F32)
        assert (cache[n, m:] == -7.0).all()
        at += m
    # the commit of the last step is what updating the pool gives
    kept = torch.tensor(lens, dtype=torch.int32, device="cuda")
    other = pool.clone()
    kda.commit_draft(cache, kept, pool, idx)
    kda.gated_decode_draft(d["x"], d["r"], d["A_log"], cu, other, idx, i=d["i"], max_steps=4, update_pool=True)
    assert torch.equal(pool, other)
    # one token a row
    d = _inputs([1] * 5, ch, dtype, seed=6)
    k = _ref(d, [1] * 5, pool[slots_of(idx, 8)])
    y = kda.gated_decode(d["x"], d["r"], d["A_log"], pool, idx, i=d["i"])
    _clean(kda.gated_decode)
    ref.check(y, k["y"], k["err"], dtype)
    ref.check(pool[slots_of(idx, 8)], k["y"], k["err"], F32)


@pytest.mark.parametrize("cu,bad", [([0, 5, 3, 40], 2), ([0, 50, 60, 40], 2), ([-1, 5, 9, 40], 2)])
def test_bad_lengths_skip_their_sequences_alone(cu, bad):
    d = _inputs([40], 36, F32, seed=1)
    h0, cut = torch.randn(3, 36, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")
    out, final = torch.full((40, 36), 9.0, device="cuda"), torch.full((3, 36), 9.0, device="cuda")
    y, f, carries = kda.gated_scan(d["x"], d["r"], d["A_log"], cut, i=d["i"], state=h0, out=out, final_state=final,
                                   output_carries=True)
    assert kda.read_device_status(kda.gated_scan.last_workspace) == bad
    dx, dr, di, da, dh = kda.gated_scan_backward(d["dy"], d["x"], d["r"], d["A_log"], cut, carries, i=d["i"],
                                                 state=h0, dfinal=h0)
    assert kda.read_device_status(kda.gated_scan_backward.last_workspace) == bad
    used = torch.zeros(40, dtype=torch.bool)
    owner = [-1] * 40
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        if 0 <= a <= b <= 40:
            used[a:b] = True
            owner[a:b] = [n] * (b - a)
        else:
            assert (f[n] == 9.0).all() and (dh[n] == 0).all()
    assert (y.cpu()[~used] == 9.0).all()
    for t in (dx, dr, di):
        assert (t.cpu()[~used] == 0).all() and torch.isfinite(t).all()
    for n, (a, b) in enumerate(zip(cu, cu[1:])):  # sequences that kept all their rows
        if 0 <= a < b <= 40 and owner[a:b] == [n] * (b - a):
            part = {key: d[key][a:b] for key in ("x", "r", "i")}
            k = ref.forward(part["x"], part["r"], part["i"], d["A_log"], [b - a], [h0[n]])
            ref.check(y[a:b], k["y"], k["err"])
            ref.check(f[n], k["final"][0], k["err"][-1])


def test_bad_slots_and_rows_of_no_sequence():
    lens = [5, 6, 7]
    d = _inputs([30], 36, BF, seed=1)
    cu = torch.tensor([2, 7, 13, 20], dtype=torch.int32, device="cuda")  # two rows before, ten behind
    pool = torch.randn(4, 36, device="cuda")
    before, out = pool.clone(), torch.full((30, 36), 9.0, device="cuda", dtype=BF)
    kda.gated_scan(d["x"], d["r"], d["A_log"], cu, i=d["i"], state=pool, out=out,
                   state_indices=torch.tensor([1, 4, -1], dtype=torch.int32, device="cuda"))
    assert kda.read_device_status(kda.gated_scan.last_workspace) == 1
    k = ref.forward(d["x"][2:20], d["r"][2:20], d["i"][2:20], d["A_log"], lens, [before[1], before[0], before[3]])
    ref.check(out[2:7], k["y"][:5], k["err"][:5], BF)
    ref.check(out[13:20], k["y"][11:], k["err"][11:], BF)
    ref.check(pool[1], k["final"][0], k["err"][4])
    assert (out[:2] == 9).all() and (out[7:13] == 9).all() and (out[20:] == 9).all()
    assert torch.equal(pool[[0, 2]], before[[0, 2]])
    y = torch.full((3, 36), 9.0, device="cuda", dtype=BF)
    kda.gated_decode(d["x"][:3], d["r"][:3], d["A_log"], pool, i=d["i"][:3], out=y,
                     state_indices=torch.tensor([0, -2, 2], dtype=torch.int32, device="cuda"))
    assert kda.read_device_status(kda.gated_decode.last_workspace) == 1 and (y[1] == 9).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_is_no_number_stays_in_its_sequence_and_channel(dtype):
    lens = [100, 150, 60, 200]
    d = _inputs(lens, 40, dtype, seed=4)
    clean = _scan(d, lens, output_carries=True)
    grads = _back(d, lens, clean[2])
    x, r, h0, dy = d["x"].clone(), d["r"].clone(), d["h0"].clone(), d["dy"].clone()
    x[120, 3], r[130, 7], h0[2, 9] = float("nan"), float("nan"), float("inf")
    dy[140, 11] = float("nan")
    e = dict(d, x=x, r=r, h0=h0, dy=dy)
    y, final, carries = _scan(e, lens, output_carries=True)
    bad = torch.zeros(510, 40, dtype=torch.bool)
    bad[120:250, 3], bad[130:250, 7], bad[250:310, 9] = True, True, True
    assert not torch.isfinite(y.cpu()[bad]).all(0).any()
    assert torch.equal(y.cpu()[~bad], clean[0].cpu()[~bad])
    assert torch.isnan(y[120:250, 3]).all() and torch.isfinite(y.cpu()[~bad]).all()
    got = _back(e, lens, carries)
    # the state's derivative flows back: from the NaN of r and dy to its sequence's first row
    hit = bad.clone()
    hit[100:250, 7], hit[100:141, 11], hit[100:250, 3] = True, True, True
    for a, b in zip(got[:3], grads[:3]):
        assert torch.equal(a.cpu()[~hit], b.cpu()[~hit])
    whole = [c for c in range(40) if c not in (3, 7, 9, 11)]
    assert torch.equal(got[3][whole], grads[3][whole])
    assert torch.isnan(got[4][1, 7]) and torch.isnan(got[4][1, 11])
    assert torch.equal(got[4][[0, 3]], grads[4][[0, 3]])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gates_at_their_ends(dtype):
    lens, ch = [90, 40], 24
    d = _inputs(lens, ch, dtype, seed=8)
    r, i, al = d["r"].clone(), d["i"].clone(), d["A_log"].clone()
    r[:, 0], r[:, 1], r[:, 2] = 200.0, -200.0, float("-inf")
    r[:, 3], i[:, 4], i[:, 5] = float("inf"), 200.0, -200.0
    al[6], al[7], al[8] = 100.0, -100.0, float("-inf")
    i[:, 9] = float("inf")
    d = dict(d, r=r, i=i, A_log=al)
    y, final, carries = _scan(d, lens, output_carries=True)
    k = _ref(d, lens)
    # |r| log2(e) 2^-24 of the fast exponential passes what the bound assumes only where the gate is shut or
    # open to the last digit; rates are bounded by the largest number
    ref.check(y, k["y"], k["err"] + 2.0 ** -30, dtype)
    got = _back(d, lens, carries)
    want, err = ref.backward(k, d["dy"], d["dfinal"], lens)
    for name, t in zip(("dx", "dr", "di", "dA_log", "dstate"), got):
        ref.check(t, torch.nan_to_num(want[name]), torch.nan_to_num(err[name]) + 2.0 ** -30,
                  dtype if name in ("dx", "dr", "di") else F32, name)


def test_differences():
    """The derivative along a direction against the difference of two forward passes in fp32.  The loss is
    a sum of products with dy and dfinal; steps of 2^-6 leave the third-order term (about 2^-12 of the size)
    and the roundings of ~1e3 terms divided by the step (2^-20 * 2^6)."""
    lens = [50, 0, 130]
    d = _inputs(lens, 32, F32, seed=12)
    y, final, carries = _scan(d, lens, output_carries=True)
    grads = _back(d, lens, carries)
    g = torch.Generator().manual_seed(1)
    names = ("x", "r", "i", "A_log", "h0")
    for name, grad in zip(names, grads):
        v = torch.randn(d[name].shape, generator=g).cuda()
        def loss(step):
            e = dict(d)
            e[name] = d[name] + step * v
            y, f = _scan(e, lens)
            return float((y.double() * d["dy"].double()).sum() + (f.double() * d["dfinal"].double()).sum())
        eps = 2.0 ** -6
        diff = (loss(eps) - loss(-eps)) / (2 * eps)
        size = float((grad.double() * v.double()).abs().sum())
        assert abs(diff - float((grad.double() * v.double()).sum())) <= 2.0 ** -11 * size, name


def test_bit_identical_from_run_to_run_and_in_a_graph():
    lens = [3000, 1, 0, 4000, 129]
    d = _inputs(lens, 256, BF, seed=11)
    cu = cu_of(lens).cuda()
    def step():
        y, f, c = kda.gated_scan(d["x"], d["r"], d["A_log"], cu, i=d["i"], state=d["h0"], output_carries=True)
        return (y, f, *kda.gated_scan_backward(d["dy"], d["x"], d["r"], d["A_log"], cu, c, i=d["i"],
                                               state=d["h0"], dfinal=d["dfinal"]))
    first = [t.clone() for t in step()]
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in out:
        t.zero_()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace (made by the call)."""
    lens = [4000, 3000]
    ds = [_inputs(lens, 512, BF, seed=s) for s in (1, 2)]
    want = [_scan(d, lens)[0] for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for d, st in zip(ds, streams):
            got.append(kda.gated_scan(d["x"], d["r"], d["A_log"], cu_of(lens).cuda(), i=d["i"], state=d["h0"],
                                      stream=st)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_wait_that_gives_up_is_reported_and_the_next_call_is_right():
    import ctypes
    lib = kda.load()
    lens = [20000]
    d = _inputs(lens, 64, BF, seed=1)
    want, _ = _scan(d, lens)
    lib.kda_set_pipeline_wait_limit(ctypes.c_uint64(1))
    try:
        _scan(d, lens)
        bits = kda.read_device_status(kda.gated_scan.last_workspace)
    finally:
        lib.kda_set_pipeline_wait_limit(ctypes.c_uint64(0))
    assert bits in (0, 4)  # on a fast enough tile nothing has to wait for long
    y, _ = _scan(d, lens)
    _clean(kda.gated_scan)
    assert torch.equal(y, want)


def test_no_rows_and_no_sequences():
    for T, N in ((0, 0), (0, 3), (4, 0)):
        x = torch.zeros(T, 16, device="cuda")
        al, cu = torch.zeros(16, device="cuda"), torch.zeros(N + 1, dtype=torch.int32, device="cuda")
        h0 = torch.randn(N, 16, device="cuda")
        y, f, c = kda.gated_scan(x, x, al, cu, i=x, state=h0, output_carries=True)
        assert y.shape == (T, 16) and torch.equal(f, h0)
        dx, dr, di, da, dh = kda.gated_scan_backward(x, x, x, al, cu, c, i=x, state=h0, dfinal=h0)
        assert torch.equal(dh, h0) and (da == 0).all() and (dx == 0).all() and dx.shape == (T, 16)


@pytest.mark.parametrize("dtype,ch", [(BF, 64), (BF, 37), (F32, 64)])
def test_rows_of_no_sequence_spread_nothing(dtype, ch):
    """NaN in the rows before and behind the sequences, in both passes: the sequences' results are those of a
    call without these rows, and the other rows' gradients are 0."""
    lens, a, b = [150, 0, 90], 61, 301
    d = _inputs(lens, ch, dtype, seed=9)
    pad = {k: torch.full((400, ch), float("nan"), dtype=dtype, device="cuda") for k in ("x", "r", "i", "dy")}
    for k, t in pad.items():
        t[a:b] = d[k]
    cu = torch.tensor([a, a + 150, a + 150, b], dtype=torch.int32, device="cuda")
    y, final, carries = kda.gated_scan(pad["x"], pad["r"], d["A_log"], cu, i=pad["i"], state=d["h0"],
                                       output_carries=True)
    got = kda.gated_scan_backward(pad["dy"], pad["x"], pad["r"], d["A_log"], cu, carries, i=pad["i"], state=d["h0"],
                                  dfinal=d["dfinal"])
    k = _ref(d, lens)
    want, err = ref.backward(k, d["dy"], d["dfinal"], lens)
    ref.check(y[a:b], k["y"], k["err"], dtype, "y")
    for name, t in zip(("dx", "dr", "di", "dA_log", "dstate"), got):
        if name in ("dx", "dr", "di"):
            assert (t[:a] == 0).all() and (t[b:] == 0).all()
            t = t[a:b]
        ref.check(t, want[name], err[name], dtype if name in ("dx", "dr", "di") else F32, name)
    assert torch.isfinite(final).all()


def test_gradients_where_no_sequence_is():
    """Rows, but no sequences: what the forward pass leaves before each 48 rows is not written then, and not used."""
    x = torch.full((100, 32), float("nan"), device="cuda")
    carries, al = torch.full((3, 32), float("nan"), device="cuda"), torch.zeros(32, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dr, di, da, dh = kda.gated_scan_backward(x, x, x, al, cu, carries, i=x)
    assert all((t == 0).all() for t in (dx, dr, di, da)) and dh is None
