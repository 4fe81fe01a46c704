"""Draws under top-k and top-p from rows that are masked down to fewer entries than top-k: the search by count finds
no k-th entry there and the search by mass comes right behind it, by every number of CTAs a row.  Tokens and
probabilities against the definition in 64 bits, as in ``test_sample_gpu``, and equal from run to run."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from tests.test_sample_gpu import BF, F32, INF, _check, _noise

pytestmark = pytest.mark.gpu


def _masked(n, vocab, left, seed):
    """Rows of normal logits, of which ``left`` (each row its own number) at random places are not masked."""
    g = torch.Generator().manual_seed(seed)
    z, noise = torch.randn(n, vocab, generator=g) * 2, _noise(n, vocab, g)
    for i in range(n):
        z[i, torch.randperm(vocab, generator=g)[left[i % len(left)]:]] = -INF
    return z, noise


@pytest.mark.parametrize("vocab", [1500, 3000, 7000, 60000, 140000])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_fewer_entries_than_top_k(vocab, dtype):
    n = 12
    z, noise = _masked(n, vocab, [1, 2, 49, 50, 51, 999, 1000, 1001, 40, 3, 700, 1200], vocab)
    z = z.to(dtype)
    k = [50, 50, 50, 50, 50, 1000, 1000, 1000, 1400, 2, 1499, 1300]
    _check(z, noise, k=k)
    _check(z, noise, k=k, top_p=[0.3 + 0.06 * i for i in range(n)])
    _check(z, noise, k=k, top_p=[0.9] * n, min_p=[0.01] * n, t=[0.5 + 0.1 * i for i in range(n)])


def test_many_rows_are_equal_from_run_to_run():
    """More clusters than fit the GPU at once, most rows with fewer entries than top-k."""
    n, vocab = 300, 40000
    z, noise = _masked(n, vocab, [30, 500, 20, 900, 45, 2000], 1)
    lg, nz, f = z.cuda(), noise.cuda(), dict(top_k=1000, top_p=0.8)
    first = kda.sample(lg, nz, **f), kda.sample_probs(lg, **f)
    for _ in range(10):
        assert torch.equal(kda.sample(lg, nz, **f), first[0])
        assert torch.equal(kda.sample_probs(lg, **f), first[1])
    few = slice(0, 24)
    _check(z[few], noise[few], k=[1000] * 24, top_p=[0.8] * 24)
