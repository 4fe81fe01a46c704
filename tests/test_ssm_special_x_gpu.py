"""NaN and infinities in the x of the state space scan: they reach the later outputs and the state of their
own value column, and nothing else (bit for bit)."""
import pytest
import torch

from tests.test_ssm_special_gpu import AT, FORMS, INF, NAN, _both, _compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("at", AT)
def test_an_x_reaches_its_column_from_its_token_on(form, value, at):
    _, _, lens, H, G, K, V = form
    for h, v in ((0, 0), (1, 37), (H - 1, V - 1)):
        r = _both(form, lambda d, a: d["x"][a + at, h, v].fill_(value))
        ry = torch.zeros(lens[1], H, V, dtype=torch.bool)
        rs = torch.zeros(H, K, V, dtype=torch.bool)
        ry[at:, h, v] = True
        rs[h, :, v] = True
        _compare(*r, ry, rs)


@pytest.mark.parametrize("form", FORMS)
def test_several_x_of_a_chunk(form):
    """Columns and tokens of both halves of a chunk, and of its neighbours."""
    _, _, lens, H, G, K, V = form
    spots = [(3, 0, 1), (40, 0, 1), (40, 0, 2), (33, 1, 5), (20, 1, 60), (70, 1, 7), (150, H - 1, 63)]

    def change(d, a):
        for t, h, v in spots:
            d["x"][a + t, h, v] = INF
    r = _both(form, change)
    ry = torch.zeros(lens[1], H, V, dtype=torch.bool)
    rs = torch.zeros(H, K, V, dtype=torch.bool)
    for t, h, v in spots:
        ry[t:, h, v] = True
        rs[h, :, v] = True
    _compare(*r, ry, rs)
