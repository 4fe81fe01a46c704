"""The convolution's backward pass against its formulas in 64 bits and against differences of the forward
pass: lengths from zero to several tiles, odd channel counts, pitched rows, final states shorter than the
taps, invalid device data, graphs.

Bounds.  z is a sum of W + 1 products, off by (W + 2) 2^-24 of its terms' magnitudes; the activation's slope
changes by at most half of that, and is itself off by at most 2^-18 (a fast exponential's 2^-20 at |z| <= 16,
times 1 + |z|); a derivative by an input is a sum of W + 1 terms of dz. A sum over tokens adds a run of them in
a row, eight runs, and those sums of the CTAs of a channel block. A run is 48 rows at most (32, rounded up to 16s)
where T / 256 + 1 CTAs are enough; else T / 8 / CTAs + 16, with 9 CTAs at least for up to 4096 channels (32 blocks of 32
lanes by four, 304 places; of one channel a lane 1024) and one for any number."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from tests._layer_ref import BF, F32, cu_of

pytestmark = pytest.mark.gpu


def _inputs(lens, ch, W, dtype, seed=0, pitch=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    z = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    wide = z(T, 2 * ch + pitch).to(dtype).cuda()
    return dict(x=wide[:, pitch:pitch + ch], dy=wide[:, pitch + ch:], w=z(ch, W, std=0.5).to(dtype).cuda(),
                b=z(ch, std=0.1).to(dtype).cuda() if bias else None, h0=z(N, W - 1, ch).to(dtype).cuda(),
                dfinal=z(N, W - 1, ch).to(dtype).cuda())


def _ref(d, silu, lens, h0=True, dfinal=True, ctas=9):
    """dx, dweight, dbias, dstate in 64 bits and a bound of each."""
    w = d["w"].double().cpu()
    ch, W = w.shape
    T, N = sum(lens), len(lens)
    outs, errs = [dict(dx=torch.zeros(T, ch, dtype=torch.float64), dweight=torch.zeros(ch, W, dtype=torch.float64),
                       dbias=torch.zeros(ch, dtype=torch.float64),
                       dstate=torch.zeros(N, W - 1, ch, dtype=torch.float64)) for _ in range(2)]
    unit, at = 2.0 ** -24, 0
    adds = max(48, T / 8 / ctas + 16) + 8 + T / 256 + 1 + 2
    for n, m in enumerate(lens):
        first = d["h0"][n].double().cpu() if h0 else torch.zeros(W - 1, ch, dtype=torch.float64)
        ext = torch.cat([first, d["x"][at:at + m].double().cpu()])
        dext, eext = torch.zeros_like(ext), torch.zeros_like(ext)
        if dfinal:
            dext[m:] = d["dfinal"][n].double().cpu()
            eext[m:] = unit * dext[m:].abs()
        if m:
            win, b = ext.unfold(0, W, 1), 0 if d["b"] is None else d["b"].double().cpu()
            z, size = (win * w).sum(-1) + b, (win * w).abs().sum(-1) + abs(b)
            dz = d["dy"][at:at + m].double().cpu()
            err = torch.zeros_like(dz)
            if silu:
                s = torch.sigmoid(z)
                err = dz.abs() * (0.5 * (W + 2) * unit * size + 2.0 ** -18)
                dz = dz * s * (1 + z * torch.sigmoid(-z))
            for j in range(W):
                dext[j:j + m] += dz * w[:, j]
                eext[j:j + m] += (err + (W + 2) * unit * dz.abs()) * w[:, j].abs()
                outs["dweight"][:, j] += (dz * ext[j:j + m]).sum(0)
                errs["dweight"][:, j] += ((err + adds * unit * dz.abs())
                                                * ext[j:j + m].abs()).sum(0)
            outs["dbias"] += dz.sum(0)
            errs["dbias"] += (err + adds * unit * dz.abs()).sum(0)
        outs["dx"][at:at + m], errs["dx"][at:at + m] = dext[W - 1:], eext[W - 1:]
        outs["dstate"][n], errs["dstate"][n] = dext[:W - 1], eext[:W - 1]
        at += m
    return outs, errs


NAMES = ("dx", "dweight", "dbias", "dstate")


def _check(got, want, err, dtype):
    for name, t in zip(NAMES, got):
        if t is None:
            continue
        t, eps = t.double().cpu(), torch.finfo(dtype if name in ("dx", "dstate") else F32).eps / 2
        limit = 1.01 * err[name] + eps * (want[name].abs() + err[name]) + 1e-37
        assert torch.isfinite(t).all(), name
        off = (t - want[name]).abs()
        assert (off <= limit).all(), (name, float((off / limit).max()))


def _back(d, lens, silu, **kw):
    kw.setdefault("state", d["h0"])
    kw.setdefault("dfinal", d["dfinal"])
    return kda.causal_conv_backward(d["dy"], d["x"], d["w"], cu_of(lens).cuda(), bias=d["b"],
                                    activation="silu" if silu else None, **kw)


LENS = [[1], [2, 1, 1, 3], [300], [0, 5, 0, 0, 129, 1, 0], [127, 1, 128, 3, 2, 2, 1, 17, 250],
        [7, 1, 8, 1, 1, 6, 2, 9, 3] * 5]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("ch,W,dtype,pitch", [(256, 4, BF, 0), (264, 3, BF, 8), (37, 4, BF, 1), (1003, 3, F32, 0),
                                              (64, 2, F32, 4), (8, 2, BF, 0), (1, 4, F32, 0), (36, 4, F32, 0)])
def test_matches_the_formulas(lens, ch, W, dtype, pitch):
    d = _inputs(lens, ch, W, dtype, seed=len(lens) + ch, pitch=pitch)
    for silu in (False, True):
        got = _back(d, lens, silu)
        assert kda.read_device_status(kda.causal_conv_backward.last_workspace) == 0
        _check(got, *_ref(d, silu, lens), dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_strips(dtype):
    """Enough rows and channels for strips of 32 tokens, sequences across their borders."""
    lens = [1000, 31, 1, 5000, 2, 0, 2500, 3, 0, 1700]
    d = _inputs(lens, 3200, 4, dtype, seed=2)
    _check(_back(d, lens, True), *_ref(d, True, lens), dtype)


@pytest.mark.parametrize("dtype,ch,pitch", [(BF, 20001, 0), (BF, 45000, 1), (F32, 20003, 0), (BF, 48000, 0), (F32, 41000, 4)])
def test_more_channels_than_ctas_fit(dtype, ch, pitch):
    """Rounds of CTAs, in every form of access."""
    lens = [70, 0, 1, 200, 3, 40]
    d = _inputs(lens, ch, 4, dtype, seed=3, pitch=pitch)
    _check(_back(d, lens, True), *_ref(d, True, lens, ctas=1), dtype)


def test_rows_of_no_sequence_spread_nothing():
    """NaN in rows before, between (an invalid sequence) and behind the sequences."""
    lens = [50, 30]
    for dtype, ch in ((BF, 64), (BF, 37), (F32, 64)):
        d = _inputs(lens, ch, 4, dtype, seed=4)
        wide = torch.full((2, 100, ch), float("nan"), dtype=dtype, device="cuda")
        wide[0, 7:87], wide[1, 7:87] = d["x"], d["dy"]
        cu = torch.tensor([7, 57, 87], dtype=torch.int32, device="cuda")
        got = kda.causal_conv_backward(wide[1], wide[0], d["w"], cu, bias=d["b"], activation="silu", state=d["h0"],
                                       dfinal=d["dfinal"])
        assert (got[0][:7] == 0).all() and (got[0][87:] == 0).all()
        _check((got[0][7:87], *got[1:]), *_ref(d, True, lens), dtype)


def test_without_states_and_bias():
    lens = [40, 3, 0, 200]
    d = _inputs(lens, 96, 4, BF, bias=False)
    got = _back(d, lens, True, state=None, dfinal=None)
    assert got[2] is None and got[3] is None
    _check(got, *_ref(d, True, lens, h0=False, dfinal=False), BF)


@pytest.mark.parametrize("cu,bad", [([0, 5, 3, 40], 2), ([2, 20, 20, 31], 0), ([0, 50, 60, 40], 2)])
def test_rows_of_no_valid_sequence_get_zero(cu, bad):
    d = _inputs([40], 36, 4, F32, seed=1)
    h0, cut = torch.randn(3, 3, 36, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")
    dx, dw, db, dh = kda.causal_conv_backward(d["dy"], d["x"], d["w"], cut, bias=d["b"], activation="silu",
                                              state=h0, dfinal=h0)
    assert kda.read_device_status(kda.causal_conv_backward.last_workspace) == bad
    used = torch.zeros(40, dtype=torch.bool)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        if 0 <= a <= b <= 40:
            used[a:b] = True
        else:
            assert (dh[n] == 0).all()
    assert (dx.cpu()[~used] == 0).all() and all(torch.isfinite(t).all() for t in (dx, dw, db))
    if not bad:  # the rows outside count nothing
        lens = [18, 0, 11]
        e = dict(d, x=d["x"][2:31], dy=d["dy"][2:31], h0=h0, dfinal=h0)
        want, err = _ref(e, True, lens)
        _check((dx[2:31], dw, db, dh), want, err, F32)


def test_differences():
    """The derivative along a direction against the difference of two forward passes in fp32: a step of 2^-6
    leaves a third-order term of about 2^-12 of the size, and the sums' roundings over the step."""
    lens = [50, 0, 2, 130]
    d = _inputs(lens, 32, 4, F32, seed=12)
    grads = _back(d, lens, True)
    g = torch.Generator().manual_seed(1)
    for name, grad in zip(("x", "w", "b", "h0"), grads):
        v = torch.randn(d[name].shape, generator=g).cuda()

        def loss(step):
            e = dict(d)
            e[name] = d[name] + step * v
            y, f = kda.causal_conv(e["x"], e["w"], cu_of(lens).cuda(), bias=e["b"], activation="silu",
                                   state=e["h0"])
            return float((y.double() * d["dy"].double()).sum() + (f.double() * d["dfinal"].double()).sum())

        eps = 2.0 ** -6
        size = float((grad.double() * v.double()).abs().sum())
        assert abs((loss(eps) - loss(-eps)) / (2 * eps) - float((grad.double() * v.double()).sum())) \
            <= 2.0 ** -11 * size, name


def test_bit_identical_and_in_a_graph():
    lens = [700, 1, 0, 300]
    d = _inputs(lens, 512, 4, BF, seed=3)
    cu = cu_of(lens).cuda()
    call = lambda: kda.causal_conv_backward(d["dy"], d["x"], d["w"], cu, bias=d["b"], activation="silu",
                                            state=d["h0"], dfinal=d["dfinal"])
    first = [t.clone() for t in call()]
    assert all(torch.equal(a, b) for a, b in zip(first, call()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_no_rows():
    h = torch.randn(2, 3, 8, device="cuda")
    x, w = torch.zeros(0, 8, device="cuda"), torch.ones(8, 4, device="cuda")
    dx, dw, db, dh = kda.causal_conv_backward(x, x, w, torch.zeros(3, dtype=torch.int32, device="cuda"), state=h,
                                              dfinal=h)
    assert dx.shape == (0, 8) and (dw == 0).all() and torch.equal(dh, h)


def test_what_is_no_number_reaches_what_it_would():
    """A NaN of x reaches dz of the tokens whose window holds it (with an activation), theirs what reads them,
    and the sums; nothing of other sequences or channels."""
    lens = [30, 40]
    d = _inputs(lens, 16, 4, F32, seed=3)
    clean = _back(d, lens, True)
    x = d["x"].clone()
    x[29, 5] = float("nan")
    got = _back(dict(d, x=x), lens, True)
    hit = torch.zeros(70, 16, dtype=torch.bool)
    hit[26:30, 5] = True
    assert torch.isnan(got[0].cpu()[hit]).all() and torch.equal(got[0].cpu()[~hit], clean[0].cpu()[~hit])
    rest = [c for c in range(16) if c != 5]
    assert torch.isnan(got[1][5]).all() and torch.equal(got[1][rest], clean[1][rest])
    assert torch.equal(got[3], clean[3])
