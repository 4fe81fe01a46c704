"""Entries far below the largest: whatever top-k or min-p keeps stands down to 2^-126 of it, through every path of the
search, although a mass (in units of 2^-44) has no digit left of it.  Against the definition in 64 bits, as in
``test_sample_gpu``; no entry lies within 2^-28 of a border of min-p."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from tests import _draw_ref as ref
from tests.test_sample_gpu import BF, F32, _check

pytestmark = pytest.mark.gpu


def _rows(n, vocab, t, dtype, seed, step=0):
    """Normal logits, and noise in proportion to p under the temperatures t, so that any entry may be drawn."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(n, vocab, generator=g) * 2.5
    z = (torch.round(z * step) / step if step else z).to(dtype)
    p = torch.stack([ref.weights(z[i], t=float(torch.tensor(t[i], dtype=F32))) for i in range(n)])
    noise = torch.empty(n, vocab).exponential_(generator=g).clamp_min(2.0 ** -20)
    return z, (p * noise).float().clamp_min(1e-38)


def test_few_entries():
    z = torch.tensor([[0.0, -40.0, -50.0, -200.0]]).repeat(6, 1)
    noise = torch.tensor([[1e25, 1.0, 1e-3, 1.0]]).repeat(6, 1)
    _check(z, noise, k=[2, 3, 4, 1, 0, 7])
    _check(z, noise, k=[2, 3, 3, 2, 0, 3], min_p=[1e-20, 1e-20, 1e-17, 1e-17, 1e-20, 1e-30])


@pytest.mark.parametrize("vocab", [700, 5000, 32003, 140000])
@pytest.mark.parametrize("dtype,step", [(F32, 0), (F32, 8), (BF, 0)])
def test_top_k_at_low_temperatures(vocab, dtype, step):
    k = [50, 2, 20, 50, 200, 400, 600, 699]
    for t in (0.05, 0.1, 0.2):
        z, noise = _rows(len(k), vocab, [t] * len(k), dtype, vocab + step, step)
        _check(z, noise, t=[t] * len(k), k=k)
        _check(z, noise, t=[t] * len(k), k=k, min_p=[1e-20, 1e-10, 0.0, 1e-14, 1e-13, 1e-30, 1e-25, 1e-5])


def _near_one(top_p, k, t, z, noise):
    """Top-p whose border lies in the last millionth of the sum.  A mass is good to 2^-28 of itself and one unit of
    2^-44, so what lies before an entry and top_p of the sum are each off by 2^-28 of the sum and 699 units at most: below
    2^-27 + 2^-33 together.  What stands lies between what does at top_p less and more that; probabilities and
    tokens are those of what stands."""
    n, slack = z.shape[0], 2.0 ** -27 + 2.0 ** -33
    f32 = lambda v: float(torch.tensor(v, dtype=F32))
    f = dict(temperature=f32(t), top_p=torch.tensor(top_p, device="cuda"),
             top_k=torch.tensor(k, dtype=torch.int32, device="cuda"))
    probs, token = kda.sample_probs(z.cuda(), **f).double().cpu(), kda.sample(z.cuda(), noise.cuda(), **f).tolist()
    for i in range(n):
        few, many = (ref.weights(z[i], t=f32(t), k=k[i], top_p=f32(top_p[i]) + d) for d in (-slack, slack))
        got = probs[i] > 0
        assert (got[few > 0]).all() and not got[many == 0].any()
        want = torch.where(got, many, 0.0)
        want = want / want.sum()
        assert ((probs[i] - want).abs() <= 2.0 ** -21 * want).all()
        assert token[i] == int(torch.argmax(torch.where(got, many / noise[i].double(), -1.0)))


@pytest.mark.parametrize("vocab", [700, 5000, 32003, 140000])
@pytest.mark.parametrize("dtype,step", [(F32, 0), (F32, 8), (BF, 0)])
def test_top_p_near_one(vocab, dtype, step):
    k = [50, 2, 20, 50, 200, 400, 600, 699]
    for t in (0.05, 0.1, 0.2):
        z, noise = _rows(len(k), vocab, [t] * len(k), dtype, vocab + step, step)
        _near_one([0.5, 0.9, 0.99, 0.999, 0.9999, 0.99999, 0.999999, 0.9999999], k, t, z, noise)


@pytest.mark.parametrize("vocab", [3000, 32003])
def test_small_min_p(vocab):
    """Borders below a mass's unit of 2^-44, and above it where it has few digits."""
    m = [1e-20, 1e-13, 2.0 ** -44, 2.0 ** -43, 1e-12, 1e-11, 1e-9, 1e-6, 1e-30, 1e-37, 1e-45, 0.0]
    t = [0.1, 0.3, 0.2, 0.25, 0.3, 0.3, 0.35, 0.4, 0.07, 0.06, 0.05, 0.05]
    z, noise = _rows(len(m), vocab, t, F32, vocab)
    for extra in (dict(), dict(k=[vocab - 1] * len(m)), dict(k=[100] * len(m)), dict(top_p=[0.999] * len(m))):
        _check(z, noise, t=t, min_p=m, **extra)
