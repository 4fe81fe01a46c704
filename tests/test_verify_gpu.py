"""Verification of drafted tokens and the commit of the accepted states.  Counts and tokens are whole
numbers: they have to be equal to the definition's in 64 bits; committed rows are copies."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api
from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu


def _inputs(lens, vocab, seed=0, near=0.5):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    logits = torch.randn(T, vocab, generator=g) * 2
    p = torch.softmax(logits, 1)
    q = torch.softmax(logits + near * torch.randn(T, vocab, generator=g), 1)
    tokens = torch.multinomial(q, 1, generator=g)[:, 0].roll(1).to(torch.int32)
    return dict(tokens=tokens.cuda(), p=p.cuda(), q=q.cuda(), u=torch.rand(T, generator=g).cuda(),
                noise=torch.empty(N, vocab).exponential_(generator=g).clamp_min(1e-30).cuda())


def _run(d, lens, **kw):
    a = kda.verify_draft(d["tokens"], d["p"], d["q"], d["u"], d["noise"], ref.cu_of(lens).cuda(), **kw)
    return [t.tolist() for t in a]


def _want(d, lens):
    return list(ref.verify(d["tokens"], d["p"], d["q"], d["u"], d["noise"], lens))


@pytest.mark.parametrize("lens", [[1], [4], [3, 1, 0, 6, 2, 40], [5] * 70, [2] * 400])
@pytest.mark.parametrize("vocab", [1, 2, 37, 4096, 32003])
def test_matches_definition(lens, vocab):
    if sum(lens) * vocab > 1 << 24:
        lens = lens[:20]
    d = _inputs(lens, vocab, seed=vocab + len(lens))
    assert _run(d, lens) == _want(d, lens)
    assert kda.read_device_status(kda.verify_draft.last_workspace) == 0
    d["q"] = None  # drafts made without drawing
    assert _run(d, lens) == _want(d, lens)


def test_acceptance_edges():
    vocab, lens = 8, [3]
    d = _inputs(lens, vocab)
    d["tokens"] = torch.tensor([0, 5, 6], dtype=torch.int32, device="cuda")
    d["p"] = torch.full((3, vocab), 0.125, device="cuda")
    d["q"] = d["p"].clone()
    d["u"] = torch.tensor([0.999, 0.999, 0.0], device="cuda")
    assert _run(d, lens)[0] == [3]           # u q < p as p == q
    d["u"][1] = 1.0                          # equality refuses; nothing is left of p - q: p is drawn from
    assert _run(d, lens) == _want(d, lens) and _run(d, lens)[0] == [2]
    d["p"][0, 5] = 0.0                       # a token the target rules out
    assert _run(d, lens)[0] == [1] and _run(d, lens) == _want(d, lens)
    d["p"][0, 5] = float("nan")              # no number accepts nothing
    assert _run(d, lens)[0] == [1]


def test_entries_that_are_never_drawn():
    vocab, lens = 4096, [1, 2]
    d = _inputs(lens, vocab)
    d["p"][0] = 0.0                          # a row that leaves nothing
    assert _run(d, lens)[1][0] == -1
    d["p"][0] = float("nan")
    assert _run(d, lens)[1][0] == -1
    d["p"][0, 77] = 1e-30
    assert _run(d, lens)[1][0] == 77
    d["p"][0, 78] = float("inf")
    assert _run(d, lens)[1][0] == 78
    d["p"][0] = -1.0
    assert _run(d, lens)[1][0] == -1


@pytest.mark.parametrize("vocab", [8, 50000, 50001])
def test_ties_go_to_the_lowest_entry(vocab):
    lens = [1, 1]
    d = _inputs(lens, vocab)
    d["p"].fill_(0.5)
    d["noise"].fill_(1.0)
    assert _run(d, lens)[1] == [0, 0]
    d["p"][1, :vocab // 2] = 0.0
    assert _run(d, lens)[1] == [0, vocab // 2]


def test_draws_in_proportion():
    """20000 draws from a known distribution: each share within 5 standard deviations."""
    n = 20000
    p = torch.tensor([0.5, 0.0, 0.3, 0.15, 0.05], device="cuda").repeat(n, 1)
    g = torch.Generator(device="cuda").manual_seed(5)
    noise = torch.empty(n, 5, device="cuda").exponential_(generator=g)
    tok = torch.zeros(n, dtype=torch.int32, device="cuda")
    _, out = kda.verify_draft(tok, p, None, torch.zeros(n, device="cuda"), noise,
                              torch.arange(n + 1, dtype=torch.int32, device="cuda"))
    share = torch.bincount(out, minlength=5).double().cpu() / n
    want = p[0].double().cpu()
    assert ((share - want).abs() <= 5 * (want * (1 - want) / n).sqrt()).all()


def test_bad_tokens_and_lengths_are_skipped_and_reported():
    lens = [3, 3, 3]
    d = _inputs(lens, 100)
    want = _want(d, lens)
    for bad in (-1, 100):
        t = d["tokens"].clone()
        t[4] = bad
        kept = torch.full((3,), 9, dtype=torch.int32, device="cuda")
        nxt = kept.clone()
        got = _run(dict(d, tokens=t), lens, num_accepted=kept, next_token=nxt)
        assert kda.read_device_status(kda.verify_draft.last_workspace) == api.KDA_DEVICE_BAD_TOKEN
        assert got == [[want[0][0], 9, want[0][2]], [want[1][0], 9, want[1][2]]]
    t = d["tokens"].clone()
    t[3] = -5  # a request's first token is not looked up
    assert _run(dict(d, tokens=t), lens) == want
    cu = torch.tensor([0, 3, 6, 10], dtype=torch.int32, device="cuda")
    kda.verify_draft(d["tokens"], d["p"], d["q"], d["u"], d["noise"], cu)
    assert kda.read_device_status(kda.verify_draft.last_workspace) == api.KDA_DEVICE_BAD_SEQLENS


@pytest.mark.parametrize("row,dtype", [((4, 64, 64), torch.float32), ((3, 40), torch.bfloat16),
                                       ((3, 37), torch.bfloat16), ((1, 5), torch.float32)])
@pytest.mark.parametrize("indexed", [False, True])
def test_commit_copies_the_accepted_step(row, dtype, indexed):
    n, steps, slots = 7, 4, 11
    wide = torch.randn(n, steps + 1, *row, device="cuda").to(dtype)
    cache = wide[:, :steps]  # requests further apart than their steps
    pool = torch.randn(slots, *row, device="cuda").to(dtype)
    kept = torch.tensor([0, 1, 4, 2, 3, 0, 4], dtype=torch.int32, device="cuda")
    idx = torch.tensor([3, 9, -1, 0, 5, 6, 2], dtype=torch.int32, device="cuda") if indexed else None
    want = pool.clone()
    for i, a in enumerate(kept.tolist()):
        s = i if idx is None else ref.slots_of(idx, slots)[i]
        if a:
            want[s] = cache[i, a - 1]
    got = kda.commit_draft(cache, kept, pool, idx)
    assert got is pool and torch.equal(pool, want)
    assert kda.read_device_status(kda.commit_draft.last_workspace) == 0


def test_commit_skips_bad_counts_and_slots():
    cache = torch.randn(4, 2, 3, 8, device="cuda")
    pool = torch.zeros(5, 3, 8, device="cuda")
    kept = torch.tensor([1, 3, -1, 2], dtype=torch.int32, device="cuda")
    kda.commit_draft(cache, kept, pool)
    assert kda.read_device_status(kda.commit_draft.last_workspace) == api.KDA_DEVICE_BAD_COUNT
    assert torch.equal(pool[0], cache[0, 0]) and torch.equal(pool[3], cache[3, 1])
    assert not pool[[1, 2, 4]].any()
    idx = torch.tensor([0, 5, -2, 1], dtype=torch.int32, device="cuda")
    kept.fill_(1)
    kda.commit_draft(cache, kept, pool, idx)
    assert kda.read_device_status(kda.commit_draft.last_workspace) == api.KDA_DEVICE_BAD_SLOT
    assert torch.equal(pool[1], cache[3, 0])
