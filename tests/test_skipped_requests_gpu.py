"""Requests that verification skips (a drafted token outside the vocabulary, bad lengths), and the commit
that follows without the host looking: nothing may be committed for them."""
import ctypes

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api, layer
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
    assert kda.read_device_status(kda.commit_draft.last_workspace) == 0
    assert kept[1].item() == 0 and nxt[1].item() == -1
    assert not pool[1].any()
    for n in (i for i in range(4) if i not in skipped):
        assert (kept[n].item(), nxt[n].item()) == (want[0][n], want[1][n])
        assert torch.equal(pool[n], cache[n, want[0][n] - 1])


def test_no_tokens_at_all_and_no_noise():
    """With no token in the batch the probabilities, tokens and noise may be missing."""
    n = 3
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    kept, nxt = (torch.full((n,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    lib, st = layer._load(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rc = lib.kda_verify_draft(n, 0, 1000, None, None, None, None, None, cu.data_ptr(), kept.data_ptr(),
                              nxt.data_ptr(), ws.data_ptr(), 256, st)
    assert rc == 0 and kda.read_device_status(ws) == 0
    assert kept.tolist() == [0] * n and nxt.tolist() == [-1] * n
