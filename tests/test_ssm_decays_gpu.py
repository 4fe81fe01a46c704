"""The tensor-core scan where steps and decays are strong, element by element.

A sequence of at most a chunk from a zero state: y = W x + D x with W[t][s] = (c_t . b_s) d_s exp(sum of
the log-decays of s+1 .. t), s <= t.  W's entries are rounded to bf16 once (2^-8 at most: 8 significant bits)
and y once more.
Their weights come from fast exponentials and logarithms (2^-20) and from a difference of running sums of
log2-decays that are kept to 32 x 256 = 2^13 (an entry below 2^-256 is zero in fp32 however it is summed):
each rounding of those is 2^-12 at most, a sum over 32 tokens in pairs takes five, two sums 10 2^-12 ln 2 =
1.7e-3 at the very worst and only where most tokens of the 32 forget everything; 2^-9 covers it.  The dot
products c_t . b_s are fp32 sums of 128 exact products: 2^-18 of the sum of their magnitudes."""
import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda
from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = ref.BF, ref.F32


def _inputs(lens, H, G, K, V, seed):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    n = lambda *s: torch.randn(*s, generator=g)
    return dict(x=n(T, H, V).to(BF), B=n(T, G, K).to(BF), C=n(T, G, K).to(BF), dt=n(T, H),
                D=n(H)), g


def _check(d, A_log, lens, with_d=True):
    dt = d["dt"].to(BF)
    c = lambda t: t.cuda()
    y, _ = kda.ssm_scan(c(d["x"]), c(dt), c(A_log), c(d["B"]), c(d["C"]), ref.cu_of(lens).cuda(),
                        D=c(d["D"]) if with_d else None)
    assert kda.read_device_status(kda.ssm_scan.last_workspace) == 0
    y = y.double().cpu()
    assert torch.isfinite(y).all()
    H, rep, a = dt.shape[1], dt.shape[1] // d["B"].shape[1], 0
    for n in lens:
        x, B, C = (d[k][a:a + n].double() for k in ("x", "B", "C"))
        z = dt[a:a + n].double()
        step = torch.logaddexp(z, torch.zeros_like(z))
        low = -torch.exp(A_log.double()) * step
        for h in range(H):
            b, cc = B[:, h // rep], C[:, h // rep]
            after = torch.ones(n, n, dtype=torch.bool).tril(-1)
            span = torch.cumsum(torch.where(after, low[:, h][:, None], 0.0), 0)
            w = torch.where(after | torch.eye(n, dtype=torch.bool), torch.exp(span), 0.0) * step[:, h]
            W, size = (cc @ b.T) * w, (cc.abs() @ b.abs().T) * w
            want = W @ x[:, h] + (d["D"].double()[h] * x[:, h] if with_d else 0)
            bound = (2.0 ** -8 + 2.0 ** -9) * (W.abs() @ x[:, h].abs()) + 2.0 ** -18 * (size @ x[:, h].abs()) \
                + 2.0 ** -8 * want.abs() * 1.01 + 1e-30
            over = (y[a:a + n, h] - want).abs() / bound
            assert float(over.max()) <= 1.0, (n, h, float(over.max()), divmod(int(over.argmax()), x.shape[-1]))
        a += n


LENS = [64, 40, 1, 33, 64]


@pytest.mark.parametrize("H,G,K,V", [(4, 1, 128, 64), (3, 1, 64, 128)])
@pytest.mark.parametrize("a_log", [2.77, 8.0, 9.0, 10.0, 12.0, 100.0])
@pytest.mark.parametrize("shift", [0.0, 3.0])
def test_decays_that_leave_the_diagonal(H, G, K, V, a_log, shift):
    """Where everything is forgotten at once y is a token's own part, whose weight is its step. (From e^89
    on the rate is no fp32 number.)"""
    d, _ = _inputs(LENS, H, G, K, V, seed=int(a_log * 10))
    d["dt"] += shift
    _check(d, torch.full((H,), a_log), LENS)


@pytest.mark.parametrize("H,G,K,V", [(4, 1, 128, 64), (3, 1, 64, 128)])
@pytest.mark.parametrize("size", [30.0, 1000.0, 30000.0])
@pytest.mark.parametrize("every", [5, 13, 31])
def test_resets_between_small_steps(H, G, K, V, size, every):
    """A huge step forgets what was before it; the tokens after it fade from it at their own small rate."""
    d, g = _inputs(LENS, H, G, K, V, seed=every)
    d["dt"] = d["dt"] * 0.5 - 5
    d["dt"][torch.arange(sum(LENS)) % every == every // 2] = size
    _check(d, torch.log(torch.rand(H, generator=g) * 15 + 1), LENS)


@pytest.mark.parametrize("dtype,core", [(BF, False), (BF, True), (F32, False)])
def test_rates_past_fp32_and_steps_of_zero(dtype, core):
    """A step of zero (a padded token) keeps the state as it is, whatever the rate; a step forgets it."""
    H, K, V, n = 4, 128, 64, 70
    d, g = _inputs([n], H, 1, K, V, seed=1)
    x, B, C = (d[k].to(dtype).cuda() for k in ("x", "B", "C"))
    h0 = torch.randn(1, H, K, V, generator=g).cuda()
    a_log = torch.tensor([100.0, 89.0, 88.0, float("inf")], device="cuda")
    dt = torch.full((n, H), -300.0, device="cuda", dtype=dtype)
    y, S = kda.ssm_scan(x, dt, a_log, B, C, ref.cu_of([n]).cuda(), state=h0, cuda_core_path=core)
    want = torch.einsum("tk,hkv->thv", C[:, 0].double(), h0[0].double())
    assert torch.equal(S, h0)
    assert ref.rel(y, want.cpu()) <= (3 * 2.0 ** -9 if dtype == BF else 2e-5)
    pool = h0.clone()
    y1 = kda.ssm_decode(x[:1], dt[:1], a_log, B[:1], C[:1], pool)
    assert torch.equal(pool, h0) and ref.rel(y1[0], want[0].cpu()) <= (3 * 2.0 ** -9 if dtype == BF else 2e-5)
    dt[n - 1] = 1.0
    _, S = kda.ssm_scan(x, dt, a_log, B, C, ref.cu_of([n]).cuda(), state=h0, cuda_core_path=core)
    step = torch.nn.functional.softplus(torch.ones((), dtype=torch.float64))
    want = step * B[-1, 0].double()[:, None] * x[-1].double()[:, None, :]
    assert ref.rel(S[0], want.cpu()) <= 2e-5
