"""Tokens and probabilities from logits against the definition in 64 bits: vocabularies of one entry to the
largest, every filter alone and together, equal values, masks, extreme parameters, rows with nothing left,
pitched and misaligned rows, graphs.

Tokens and which entries stand have to be equal: sums are exact to 2^-28 of an entry, and the inputs are
fixed ones whose borders lie further apart.  Probabilities are one fp32 quotient of p (relative error 2^-22:
its series, its table entry, a product) and a sum, rounded three times: 2^-21."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from tests import _draw_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def _noise(n, vocab, g):
    return torch.empty(n, vocab).exponential_(generator=g).clamp_min(1e-30)


def _check(logits, noise, **params):
    """Token and probabilities of every row; ``params`` lists of one value a row."""
    n = logits.shape[0]
    rows = [dict(zip(params, v)) for v in zip(*params.values())] if params else [{}] * n
    names = dict(t="temperature", k="top_k", top_p="top_p", min_p="min_p")
    dev = {names[p]: torch.tensor(v, dtype=torch.int32 if p == "k" else F32, device="cuda") for p, v in params.items()}
    f32 = lambda x: float(torch.tensor(x, dtype=F32))
    rows = [{p: v if p == "k" else f32(v) for p, v in r.items()} for r in rows]
    lg, nz = logits.cuda(), noise.cuda()
    token = kda.sample(lg, nz, **dev).tolist()
    probs = kda.sample_probs(lg, **dev).double().cpu()
    bad = any(not r.get("t", 1) >= 0 or r.get("top_p", 1) != r.get("top_p", 1) or r.get("min_p", 0) != r.get("min_p", 0)
              for r in rows)
    for fn in (kda.sample, kda.sample_probs):
        assert kda.read_device_status(fn.last_workspace) == (0x40 if bad else 0)
    for i, r in enumerate(rows):
        w = ref.weights(logits[i], **r)
        w = torch.where(w < 2.0 ** -126, 0.0, w)
        want = w / w.sum() if bool((w > 0).any()) else w
        assert torch.equal(probs[i] > 0, want > 2.0 ** -149), (i, r, (probs[i] > 0).sum(), (want > 0).sum())
        assert ((probs[i] - want).abs() <= 2.0 ** -21 * want + 2.0 ** -149).all(), (i, r)
        assert token[i] == ref.token(logits[i], noise[i], **r), (i, r)


@pytest.mark.parametrize("vocab", [1, 2, 31, 500, 4097, 32003, 131072, 151936, 360448])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_filters_alone_and_together(vocab, dtype):
    g = torch.Generator().manual_seed(vocab)
    n = 9 if vocab < 100000 else 5
    logits, noise = (torch.randn(n, vocab, generator=g) * 2.5).to(dtype), _noise(n, vocab, g)
    t = [0.3 + 0.2 * i for i in range(n)]
    k = [0, 1, 2, 5, 40, 1000, vocab - 1, vocab, 1 << 30][-n:] if n == 5 else [0, 1, 2, 5, 40, 1000, vocab - 1, vocab, 7]
    tp = [0.9, 0.05, 0.5, 0.99, 1.0, 0.999, 0.0, 0.7, 0.95][:n]
    mp = [0.0, 0.5, 0.01, 1.0, 0.1, 0.001, 0.2, 2.0, 1e-6][:n]
    _check(logits, noise)
    _check(logits, noise, t=t)
    _check(logits, noise, k=k)
    _check(logits, noise, top_p=tp)
    _check(logits, noise, min_p=mp)
    _check(logits, noise, t=t, k=k, top_p=tp[::-1], min_p=mp)
    _check(logits, noise, t=[0.0, 1.0] * (n // 2) + [0.0], top_p=tp)


@pytest.mark.parametrize("vocab", [3000, 140000])
def test_equal_values(vocab):
    """Rows of one value, of two, of few: the order by index decides, over more equal entries than are
    ranked at once."""
    g = torch.Generator().manual_seed(1)
    z = torch.randn(6, vocab, generator=g)
    z[0], z[1] = 2.5, (torch.arange(vocab) % 2).float()
    z[2] = torch.round(z[2])
    z[3] = torch.where(torch.arange(vocab) % 7 == 3, 0.0, -0.0)
    z[4] = torch.round(z[4] * 4) / 4
    z[5] = torch.where(z[5] > 0, 0.0, z[5] * 1e-30)          # values a hair apart
    noise = _noise(6, vocab, g)
    for f in (dict(k=[17, vocab // 2 + 5, 1500, vocab - 2, 2900, 2000]), dict(top_p=[0.3, 0.8, 0.5, 0.001, 0.9, 0.99]),
              dict(k=[2999] * 6, top_p=[0.7] * 6), dict(min_p=[1.0] * 6), dict(t=[0.0] * 6)):
        _check(z, noise, **f)


def test_masks_and_what_is_no_number():
    vocab = 5000
    g = torch.Generator().manual_seed(2)
    z, noise = torch.randn(10, vocab, generator=g) * 2, _noise(10, vocab, g)
    low = torch.finfo(F32).min
    z[0, :4990], z[1, 5:] = -INF, low            # few entries left
    z[2] = low                                   # all at the type's lowest value: all alike
    z[3] = -INF                                  # nothing left
    z[4] = NAN
    z[5, ::3] = NAN
    z[6, 100], z[6, 4000], z[6, 7] = INF, INF, NAN
    z[7, 0], z[7, 1] = torch.finfo(F32).max, low
    z[8, :], z[8, 17] = -INF, -5.0
    z[9] = INF
    for f in (dict(), dict(k=[50] * 10), dict(top_p=[0.9] * 10), dict(t=[0.5] * 10, k=[60] * 10, top_p=[0.8] * 10,
              min_p=[0.05] * 10), dict(t=[0.0] * 10)):
        _check(z, noise, **f)


def test_parameters_at_their_ends():
    vocab, n = 4000, 12
    g = torch.Generator().manual_seed(3)
    z, noise = torch.randn(n, vocab, generator=g) * 3, _noise(n, vocab, g)
    _check(z, noise, t=[-1.0, NAN, INF, 1e-30, 1e30, 1e-3, 100.0, 0.0, 1.0, 1.0, 1.0, 1.0],
           top_p=[1.0, 1.0, 0.5, 0.5, 0.5, 0.9, 0.9, 0.9, NAN, -1.0, 1e-30, 5.0],
           min_p=[0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, NAN],
           k=[0, 0, 0, 0, 0, 0, -5, 0, 0, 0, 3, 0])


def test_numbers_for_all_rows_and_pitched_rows():
    g = torch.Generator().manual_seed(4)
    wide, noise = torch.randn(7, 1501, generator=g) * 2, _noise(7, 1400, g)
    for dtype, off in ((F32, 0), (F32, 1), (BF, 1), (BF, 0)):
        lg = wide.to(dtype).cuda()[:, off:off + 1299]
        nz = noise.cuda()[:, 3:1302]
        f = dict(temperature=0.75, top_k=50, top_p=0.5, min_p=0.125)
        token, probs = kda.sample(lg, nz, **f), kda.sample_probs(lg, **f)
        for i in range(7):
            w = ref.weights(lg[i], t=0.75, k=50, top_p=0.5, min_p=0.125)
            want = w / w.sum()
            assert ((probs[i].double().cpu() - want).abs() <= 2.0 ** -21 * want).all()
            assert int(token[i]) == ref.token(lg[i], nz[i], t=0.75, k=50, top_p=0.5, min_p=0.125)


def test_outputs_given_a_graph_and_no_rows():
    g = torch.Generator().manual_seed(5)
    z, noise = (torch.randn(70, 33000, generator=g) * 2).cuda(), _noise(70, 33000, g).cuda()
    t, p = torch.rand(70, device="cuda") + 0.5, torch.rand(70, device="cuda")
    token, probs = torch.empty(70, dtype=torch.int32, device="cuda"), torch.empty(70, 33000, device="cuda")
    assert kda.sample(z, noise, temperature=t, top_p=p, out=token) is token
    assert kda.sample_probs(z, temperature=t, top_p=p, out=probs) is probs
    first = token.clone(), probs.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.sample(z, noise, temperature=t, top_p=p, out=token)
        kda.sample_probs(z, temperature=t, top_p=p, out=probs)
    for _ in range(3):
        token.zero_()
        probs.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(token, first[0]) and torch.equal(probs, first[1])
    # the token is a draw from the probabilities
    assert torch.equal(torch.argmax(probs / noise, 1).int(), token)
    assert kda.sample(z[:0], noise[:0]).shape == (0,) and kda.sample_probs(z[:0]).shape == (0, 33000)


def test_verification_takes_the_probabilities():
    """Drafts drawn with the same logits as the target's are kept throughout; the row after the last is a
    draw of its own."""
    g = torch.Generator().manual_seed(6)
    n, drafts, vocab = 5, 3, 2000
    z = (torch.randn(n * (drafts + 1), vocab, generator=g) * 2).cuda()
    f = dict(temperature=0.8, top_k=40, top_p=0.9)
    probs = kda.sample_probs(z, **f)
    noise = _noise(n * (drafts + 1), vocab, g).cuda()
    drawn = kda.sample(z, noise, **f).view(n, drafts + 1)
    tokens = torch.cat([torch.zeros(n, 1, dtype=torch.int32, device="cuda"), drawn[:, :drafts]], 1).flatten()
    cu = torch.arange(0, n * (drafts + 1) + 1, drafts + 1, dtype=torch.int32, device="cuda")
    last = torch.arange(drafts, n * (drafts + 1), drafts + 1, device="cuda")
    kept, token = kda.verify_draft(tokens, probs, probs, torch.rand(n * (drafts + 1), device="cuda") * 0.999,
                                   noise[last].contiguous(), cu)
    assert (kept == drafts + 1).all() and torch.equal(token, drawn[:, drafts].contiguous())


@pytest.mark.parametrize("vocab", [700, 5000, 60000])
def test_counts_around_the_number_that_is_ranked_at_once(vocab):
    """top-k from below to above the few hundred entries that are ranked by number and mass at once, over values
    of their own and over equal ones, alone and with the other filters."""
    g = torch.Generator().manual_seed(vocab)
    k = [2, 255, 300, 480, 505, 511, 512, 513, 530, 650, 699, 700]
    n = len(k)
    noise = _noise(n, vocab, g)
    z = torch.randn(n, vocab, generator=g) * 2
    for logits in (z, torch.round(z * 8) / 8, torch.where(z > 1.0, z, torch.full_like(z, -INF))):
        _check(logits, noise, k=k)
        _check(logits, noise, k=k, top_p=[0.3 + 0.06 * i for i in range(n)])
        _check(logits, noise, k=k, top_p=[0.9] * n, min_p=[0.002 * i for i in range(n)], t=[1.5 - 0.1 * i for i in range(n)])


@pytest.mark.parametrize("vocab", [1999, 4001, 8190])
def test_counts_around_what_fewer_ctas_rank_at_once(vocab):
    """One, two and four CTAs a row rank fewer entries at once, as each has more pairs to look at: top-k around 181, 256
    and 362, the square roots of 64 x 512 pairs of each."""
    g = torch.Generator().manual_seed(vocab)
    k = [170, 180, 181, 182, 200, 254, 256, 257, 350, 361, 363, 400]
    n = len(k)
    noise = _noise(n, vocab, g)
    z = torch.randn(n, vocab, generator=g) * 2
    for logits in (z, torch.round(z * 4) / 4):
        _check(logits, noise, k=k)
        _check(logits, noise, k=k, top_p=[0.4 + 0.05 * i for i in range(n)], min_p=[0.0, 0.01] * (n // 2))
