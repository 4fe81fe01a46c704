"""The tensor-core scan where its scheduling can go wrong: cuts of long sequences, workspaces of every
size, odd head counts, waits that run out, capture in a graph, repeated and interleaved calls."""
import time

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from linear_attention_prefill_chunked_gb300 import api, layer
from tests import _layer_ref as ref
from tests.test_ssm_gpu import S_BOUND, Y_BOUND, _close, _inputs, _scan, _want

pytestmark = pytest.mark.gpu
BF, F32 = ref.BF, ref.F32


def _plan_size(lens, H, G, K, V, sdt):
    return kda.ssm_scan_workspace_size(layer.ssm_desc(len(lens), sum(lens), H, G, K, V, BF, sdt))


# sequences that are cut alone, beside short and empty ones, one chunk too few to be cut, and ragged ends
CUTS = [[2600], [5, 0, 2500, 64, 1], [2000, 2001, 30], [1793, 1792], [3000] + [17] * 40]


@pytest.mark.parametrize("lens", CUTS)
@pytest.mark.parametrize("H,G,K,V", [(2, 1, 128, 64), (1, 1, 64, 128), (3, 1, 64, 64)])
@pytest.mark.parametrize("sdt", [F32, BF])
def test_cut_sequences(lens, H, G, K, V, sdt):
    d = _inputs(lens, H, G, K, V, BF, seed=sum(lens) + H, a_max=1.5, sdt=sdt)
    d["dt"] -= 3  # a memory of some hundred tokens
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    y, fin = _scan(d, lens, state=d["h0"])
    assert kda.read_device_status(kda.ssm_scan.last_workspace) == 0
    _close(y, fin, want, wfin, lens, BF, sdt)
    # in place in a pool, where the last part overwrites what the first one starts from
    N = len(lens)
    idx = torch.randperm(N + 2)[:N].to(torch.int32).cuda()
    pool = torch.zeros(N + 3, H, K, V, device="cuda", dtype=sdt)
    pool[idx.long()] = d["h0"]
    yp, _ = _scan(d, lens, state=pool, state_indices=idx)
    assert torch.equal(yp, y) and torch.equal(pool[idx.long()], fin)


@pytest.mark.parametrize("memory", ["endless", "short", "none", "padded"])
@pytest.mark.parametrize("H,G,K,V", [(3, 1, 128, 64), (1, 1, 128, 128)])
def test_cut_memories(memory, H, G, K, V):
    """Parts whose decay is hardly any, whose decay leaves nothing, and with most steps at zero."""
    lens = [4500, 1500, 70]
    d = _inputs(lens, H, G, K, V, BF, seed=H + 90, a_max=1.5)
    if memory == "endless":
        d["dt"] -= 7  # 4500 tokens keep some 0.9 of the first
        d["h0"].zero_()
    elif memory == "short":
        d["dt"] += 2
    elif memory == "none":  # decays below the smallest fp32 number within a few tokens
        d["dt"] += 40
    else:  # steps of zero, as of padded tokens: softplus underflows
        d["dt"][torch.rand(sum(lens), generator=torch.Generator().manual_seed(1)).cuda() < 0.7] = -300
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    y, fin = _scan(d, lens, state=d["h0"])
    assert kda.read_device_status(kda.ssm_scan.last_workspace) == 0
    assert ref.rel(y, want) <= Y_BOUND[BF]
    for i, n in enumerate(lens):
        # every sum of 16 tokens' products, in three parts, is cut off to 24 bits once more
        adds = 3 * (n + 15) // 16
        for h in range(H):
            e = ref.rel(fin[i, h], wfin[i][h])
            assert e <= 1.5 * S_BOUND[F32] + adds * 2.0 ** -23, (i, h, e)


def test_every_workspace_size_gives_the_same_up_to_rounding():
    lens, H, G, K, V = [2500, 40], 2, 1, 128, 64
    d = _inputs(lens, H, G, K, V, BF, seed=4, a_max=1.5)
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    full = _plan_size(lens, H, G, K, V, F32)
    for size in (256, 1024, full - 1, full, full + 4096):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # its contents do not matter
        y, fin = _scan(d, lens, state=d["h0"], workspace=ws)
        assert kda.read_device_status(ws) == 0
        _close(y, fin, want, wfin, lens, BF, F32, size)
        y2, fin2 = _scan(d, lens, state=d["h0"], workspace=ws)
        assert torch.equal(y, y2) and torch.equal(fin, fin2)


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (10, 2), (5, 5), (152, 8)])
def test_odd_heads_of_64(H, G):
    """Two heads of a group share an item; the odd one of a group is alone in its own."""
    lens = [100, 64, 7]
    d = _inputs(lens, H, G, 128, 64, BF, seed=H)
    y, fin = _scan(d, lens, state=d["h0"])
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    _close(y, fin, want, wfin, lens, BF, F32)


@pytest.mark.parametrize("lens", [[2600, 300, 5], [200] * 30])
def test_waits_that_run_out_set_the_status_and_return(lens):
    d = _inputs(lens, 4, 1, 128, 64, BF, seed=51)
    torch.cuda.synchronize()
    api.set_pipeline_wait_limit(1)
    try:
        t0 = time.perf_counter()
        _scan(d, lens, state=d["h0"])
        bits = kda.read_device_status(kda.ssm_scan.last_workspace)  # synchronises
        took = time.perf_counter() - t0
    finally:
        api.set_pipeline_wait_limit(0)
    assert bits & api.KDA_DEVICE_PIPE_TIMEOUT
    assert took < 1.5, took  # the drains found what they waited for
    y, fin = _scan(d, lens, state=d["h0"])
    assert kda.read_device_status(kda.ssm_scan.last_workspace) == 0
    want, wfin, _ = _want(d, lens, list(d["h0"]))
    _close(y, fin, want, wfin, lens, BF, F32)


def test_graph_replay_follows_its_inputs():
    lens = [1900, 70]
    d = _inputs(lens, 4, 1, 128, 64, BF, seed=61)
    cu = ref.cu_of(lens).cuda()
    run = lambda: kda.ssm_scan(d["x"], d["dt"], d["A_log"], d["B"], d["C"], cu, D=d["D"],
                               dt_bias=d["dt_bias"], state=d["h0"])
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, fin = run()
    for seed in (62, 63):
        e = _inputs(lens, 4, 1, 128, 64, BF, seed=seed)
        for n in ("x", "dt", "B", "C", "h0"):
            d[n].copy_(e[n])
        g.replay()
        wy, wf = run()
        assert torch.equal(y, wy) and torch.equal(fin, wf)


def test_two_streams_do_not_disturb_each_other():
    lens = [500, 33, 1900]
    a, b = _inputs(lens, 4, 1, 128, 64, BF, seed=71), _inputs(lens, 4, 2, 64, 64, BF, seed=72)
    wa, wb = _scan(a, lens, state=a["h0"]), _scan(b, lens, state=b["h0"])
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((_scan(a, lens, state=a["h0"], stream=sa), _scan(b, lens, state=b["h0"], stream=sb)))
    torch.cuda.synchronize()
    for ra, rb in got:
        for x, y in zip(ra + rb, wa + wb):
            assert torch.equal(x, y)


def test_large_offsets():
    """A pool whose slots lie more than 2^31 elements apart from its start."""
    H, K, V = 4, 128, 128
    stride = 1 << 28
    need = 9 * stride * 4
    if torch.cuda.mem_get_info()[0] < need * 1.2:
        pytest.skip("not enough device memory")
    lens = [65, 3]
    d = _inputs(lens, H, 1, K, V, BF, seed=81)
    flat = torch.zeros(9 * stride, device="cuda")
    pool = flat.view(9, stride)
    idx = torch.tensor([8, 0], dtype=torch.int32, device="cuda")
    for i, s in enumerate(idx.tolist()):
        pool[s, :H * K * V] = d["h0"][i].flatten()
    want, wf = _scan(d, lens, state=d["h0"])
    y, _ = _scan(d, lens, state=pool, state_indices=idx, slot_stride=stride)
    assert torch.equal(y, want)
    for i, s in enumerate(idx.tolist()):
        assert torch.equal(pool[s, :H * K * V].view(H, K, V), wf[i])
