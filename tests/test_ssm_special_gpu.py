"""NaN and infinities in the state space scan: what they must reach (their own head's, value column's or
group's later outputs and state) and what they must not (other heads and columns, earlier tokens).  What
must not be reached is compared bit for bit with the run without them."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from tests import _layer_ref as ref
from tests.test_ssm_gpu import _inputs, _scan

pytestmark = pytest.mark.gpu
BF, F32 = ref.BF, ref.F32
NAN, INF = float("nan"), float("inf")

# bf16 on the tensor cores, whole and cut, with two 64-wide heads a product and with one head of 128
FORMS = [(BF, False, [70, 200, 3], 4, 1, 128, 64), (BF, False, [70, 200], 3, 1, 64, 64),
         (BF, False, [70, 200, 3], 4, 2, 128, 128), (BF, False, [40, 2600], 2, 1, 128, 64),
         (BF, False, [40, 2600], 2, 1, 64, 128), (BF, True, [70, 200, 3], 4, 1, 128, 64),
         (F32, False, [70, 200, 3], 4, 1, 128, 64)]
AT = [0, 5, 31, 32, 63, 64, 100, 199]  # tokens of the second sequence


def _both(form, change):
    dtype, core, lens, H, G, K, V = form
    d = _inputs(lens, H, G, K, V, dtype, seed=17, a_max=2.0)
    d["dt"] -= 2
    a, b = lens[0], lens[0] + lens[1]
    y0, s0 = _scan(d, lens, state=d["h0"], cuda_core_path=core)
    change(d, a)
    y1, s1 = _scan(d, lens, state=d["h0"], cuda_core_path=core)
    assert kda.read_device_status(kda.ssm_scan.last_workspace) == 0
    assert torch.isfinite(y0.float()).all() and torch.isfinite(s0).all()
    return a, b, y0.cpu(), s0.cpu(), y1.cpu(), s1.cpu()


def _compare(a, b, y0, s0, y1, s1, reached_y, reached_s):
    """reached_y [tokens of the second sequence, H, V] and reached_s [H, K, V]: where the result has to
    be no number; everywhere else it has to be the other run's."""
    ry = torch.zeros_like(y0, dtype=torch.bool)
    ry[a:b] = reached_y
    rs = torch.zeros_like(s0, dtype=torch.bool)
    rs[1] = reached_s
    assert not torch.isfinite(y1.float())[ry].any()
    assert not torch.isfinite(s1)[rs].any()
    assert torch.equal(torch.where(ry, 0, y1), torch.where(ry, 0, y0))
    assert torch.equal(torch.where(rs, 0, s1), torch.where(rs, 0, s0))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("at", AT)
def test_a_step_reaches_its_head_from_its_token_on(form, value, at):
    _, _, lens, H, G, K, V = form
    for h in (0, 1, H - 1):
        r = _both(form, lambda d, a: d["dt"][a + at, h].fill_(value))
        ry = torch.zeros(lens[1], H, V, dtype=torch.bool)
        rs = torch.zeros(H, K, V, dtype=torch.bool)
        ry[at:, h] = True
        rs[h] = True
        _compare(*r, ry, rs)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("name", ["B", "C"])
@pytest.mark.parametrize("at", [0, 33, 64, 199])
def test_b_and_c_reach_their_group(form, name, at):
    _, _, lens, H, G, K, V = form
    k = 11
    r = _both(form, lambda d, a: d[name][a + at, G - 1, k].fill_(NAN))
    ry = torch.zeros(lens[1], H, V, dtype=torch.bool)
    rs = torch.zeros(H, K, V, dtype=torch.bool)
    heads = slice((G - 1) * (H // G), H)
    if name == "B":  # that row of the group's states from then on
        ry[at:, heads] = True
        rs[heads, k] = True
    else:            # that token's outputs
        ry[at, heads] = True
    _compare(*r, ry, rs)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("name", ["A_log", "dt_bias"])
def test_a_heads_parameters_reach_that_head(form, name):
    dtype, core, lens, H, G, K, V = form
    d = _inputs(lens, H, G, K, V, dtype, seed=19, a_max=2.0)
    y0, s0 = _scan(d, lens, state=d["h0"], cuda_core_path=core)
    for h in (0, 1):
        p = d[name].clone()
        p[h] = NAN
        y1, s1 = _scan(dict(d, **{name: p}), lens, state=d["h0"], cuda_core_path=core)
        rest = [i for i in range(H) if i != h]
        assert torch.equal(y1[:, rest], y0[:, rest]) and torch.equal(s1[:, rest], s0[:, rest])
        assert not torch.isfinite(y1[:, h].float()).any() and not torch.isfinite(s1[:, h]).any()


@pytest.mark.parametrize("form", FORMS)
def test_an_initial_state_reaches_its_row_and_column(form):
    """S[k, v] reaches the outputs of column v of its head, and stays where it is in the state."""
    dtype, core, lens, H, G, K, V = form

    def change(d, a):
        d["h0"][1, 1, 3, 9] = NAN
    r = _both(form, change)
    ry = torch.zeros(lens[1], H, V, dtype=torch.bool)
    rs = torch.zeros(H, K, V, dtype=torch.bool)
    ry[:, 1, 9] = True
    rs[1, 3, 9] = True
    _compare(*r, ry, rs)
