"""Requests that verification skips (a drafted token outside the vocabulary, bad lengths), and the commit
that follows without the host looking: nothing may be committed for them."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api
from tests import _layer_ref as ref
from tests.test_verify_gpu import _inputs, _want

pytestmark = pytest.mark.gpu


def _leave(value, n):
    """Fills what the allocator hands out next for small int32 tensors."""
    made = [torch.full((n,), value, dtype=torch.int32, device="cuda") for _ in range(8)]
    del made


@pytest.mark.parametrize("what", ["token", "lengths"])
def test_skipped_requests_commit_nothing(what):
    lens = [3, 3, 3, 2]
    d = _inputs(lens, 100)
    want = _want(d, lens)
    cu = ref.cu_of(lens).cuda()
    skipped = [1]
    if what == "token":
        d["tokens"][5] = 100
    else:
        cu[2] = 2  # request 1 runs backwards; request 2 then starts earlier
        skipped = [1, 2]
    cache = torch.randn(4, 3, 5, 8, device="cuda")
    pool = torch.zeros(4, 5, 8, device="cuda")
    _leave(2, 4)
    kept, nxt = kda.verify_draft(d["tokens"], d["p"], d["q"], d["u"], d["noise"], cu)
    assert kda.read_device_status(kda.verify_draft.last_workspace) == (
        api.KDA_DEVICE_BAD_TOKEN if what == "token" else api.KDA_DEVICE_BAD_SEQLENS)
    kda.commit_draft(cache, kept, pool)
    status = kda.read_device_status(kda.commit_draft.last_workspace)
    # request 2 of the bad lengths has 7 tokens, and may keep more than the 3 steps of the cache
    assert status == 0 or what == "lengths" and status == api.KDA_DEVICE_BAD_COUNT
    assert kept[1].item() == 0 and nxt[1].item() == -1
    assert not pool[1].any()
    for n in (i for i in range(4) if i not in skipped):
        assert (kept[n].item(), nxt[n].item()) == (want[0][n], want[1][n])
        assert torch.equal(pool[n], cache[n, want[0][n] - 1])


@pytest.mark.parametrize("mark", [None, False, True])
def test_given_outputs_are_marked_on_request(mark):
    """What a round before left in a caller's own buffers stays, or is replaced where asked for."""
    lens = [3, 3, 3]
    d = _inputs(lens, 100)
    want = _want(d, lens)
    d["tokens"][5] = -7
    kept, nxt = (torch.full((3,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
    got = kda.verify_draft(d["tokens"], d["p"], d["q"], d["u"], d["noise"], ref.cu_of(lens).cuda(),
                           num_accepted=kept, next_token=nxt, mark_skipped=mark)
    assert got[0] is kept and got[1] is nxt
    assert kept.tolist() == [want[0][0], 0 if mark else 9, want[0][2]]
    assert nxt.tolist() == [want[1][0], -1 if mark else 9, want[1][2]]
    # one given, one made
    kept.fill_(9)
    _, made = kda.verify_draft(d["tokens"], d["p"], d["q"], d["u"], d["noise"], ref.cu_of(lens).cuda(),
                               num_accepted=kept, mark_skipped=mark)
    assert kept.tolist() == [want[0][0], 0 if mark else 9, want[0][2]]
    assert made.tolist() == [want[1][0], -1, want[1][2]]
