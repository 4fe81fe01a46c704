"""Commit into pools whose slots lie further apart than a row, as the draft steps take them."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api
from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("row,dtype,stride", [((4, 16, 8), torch.float32, 640),    # 16 bytes at a time
                                              ((3, 40), torch.bfloat16, 128),
                                              ((3, 37), torch.bfloat16, 130),     # element by element
                                              ((2, 5), torch.float32, 11)])
@pytest.mark.parametrize("indexed", [False, True])
def test_padded_pool(row, dtype, stride, indexed):
    n, steps, slots = 5, 3, 7
    size = torch.Size(row).numel()
    cache = torch.randn(n, steps, *row, device="cuda").to(dtype)
    kept = torch.tensor([0, 1, 3, 2, 3], dtype=torch.int32, device="cuda")
    idx = torch.tensor([3, 5, -1, 0, 2], dtype=torch.int32, device="cuda") if indexed else None
    pool = torch.randn(slots, stride, device="cuda").to(dtype)
    want = pool.clone()
    for i, a in enumerate(kept.tolist()):
        if a:
            want[i if idx is None else ref.slots_of(idx, slots)[i], :size] = cache[i, a - 1].flatten()
    got = kda.commit_draft(cache, kept, pool, idx, slot_stride=stride)
    assert got is pool and torch.equal(pool, want)  # the padding between slots too
    assert kda.read_device_status(kda.commit_draft.last_workspace) == 0
    bad = torch.tensor([0, slots, -2, 1, 2], dtype=torch.int32, device="cuda")
    kda.commit_draft(cache, kept, pool, bad, slot_stride=stride)
    assert kda.read_device_status(kda.commit_draft.last_workspace) == api.KDA_DEVICE_BAD_SLOT


def test_drafted_from_and_committed_to_a_padded_pool():
    """The round of a serving loop on one padded pool: draft steps read it, the commit writes it."""
    H, G, K, V, lens = 4, 1, 64, 64, [3, 2]
    stride, size = H * K * V + 64, H * K * V
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=g).cuda()
    T = sum(lens)
    x, dt, B, C = n(T, H, V), n(T, H), n(T, G, K), n(T, G, K)
    a = torch.zeros(H, device="cuda")
    idx = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    padded, packed = torch.zeros(3, stride, device="cuda"), torch.zeros(3, H, K, V, device="cuda")
    kept = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    for _ in range(2):
        ca, cb = (torch.zeros(2, 3, H, K, V, device="cuda") for _ in range(2))
        ya = kda.ssm_decode_draft(x, dt, a, B, C, ref.cu_of(lens).cuda(), packed, idx, cache=ca, max_steps=3)
        yb = kda.ssm_decode_draft(x, dt, a, B, C, ref.cu_of(lens).cuda(), padded, idx, cache=cb, max_steps=3,
                                  slot_stride=stride)
        assert torch.equal(ya, yb) and torch.equal(ca, cb)
        kda.commit_draft(ca, kept, packed, idx)
        kda.commit_draft(cb, kept, padded, idx, slot_stride=stride)
        assert torch.equal(padded[:, :size].view(3, H, K, V), packed)


def test_refusals():
    cache = torch.zeros(2, 3, 4, 8, device="cuda")
    kept = torch.zeros(2, dtype=torch.int32, device="cuda")
    z = lambda *s: torch.zeros(*s, device="cuda")
    for pool, stride in ((z(3, 40), 31), (z(3, 40), -40), (z(3, 30), 40), (z(0, 40), 40), (z(40, 3).T, 40)):
        with pytest.raises(ValueError):
            kda.commit_draft(cache, kept, pool, slot_stride=stride)
    with pytest.raises(TypeError):
        kda.commit_draft(cache, kept, torch.zeros(3, 40, device="cuda").bfloat16(), slot_stride=40)
