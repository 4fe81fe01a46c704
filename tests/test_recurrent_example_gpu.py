"""The example that trains and serves the recurrent block: its gradients against the same model in elementary
operations and 64 bits, its tokens from pools against its prompts, and that it runs.

Bounds: activations pass six matrix products of 256 terms and the recurrences in fp32, each off by at most a few
2^-24 sqrt(256) of its size, backward as often: 2^-13 of a gradient's norm is above all of them, and a
wrong tap, gate, state or sequence is off by the order of the gradient itself.  fp32 products must not be
rounded to fewer bits for that."""
import os
import sys

import pytest
import torch

import linear_attention_prefill_chunked_gb300 as kda

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _plain_loss(p, tokens, after, cu, VOCAB, HID, W):
    """The model's loss token by token in 64 bits (CPU), from parameters ``p``."""
    x = p["emb"][tokens]
    out = []
    for a, b in zip(cu, cu[1:]):
        ext = torch.cat([p["conv_h0"], x[a:b]])
        h = p["h0"]
        for t in range(b - a):
            z = (ext[t:t + W] * p["conv_w"].T).sum(0) + p["conv_b"]
            u = z * torch.sigmoid(z)
            r, i = (p["gates"] @ u).split(HID)
            g = -torch.exp(p["A_log"]) * torch.sigmoid(r)
            h = torch.exp(g) * h + torch.sqrt(-torch.expm1(2 * g)) * torch.sigmoid(i) * u
            out.append(p["head"] @ (x[a + t] + p["out"] @ h))
    return torch.nn.functional.cross_entropy(torch.stack(out), after)


def test_gradients():
    import recurrent_training as ex
    torch.backends.cuda.matmul.allow_tf32 = False
    model = ex.Model(seed=3)
    tokens, after, cu = ex.batch([9, 0, 1, 70, 3], seed=5)
    loss = torch.nn.functional.cross_entropy(model(tokens, cu), after)
    loss.backward()
    assert kda.read_device_status(kda.gated_scan_backward.last_workspace) == 0
    assert kda.read_device_status(kda.causal_conv_backward.last_workspace) == 0
    p = {n: q.detach().double().cpu().requires_grad_() for n, q in model.named_parameters()}
    want = _plain_loss(p, tokens.long().cpu(), after.cpu(), cu.tolist(), ex.VOCAB, ex.HID, ex.W)
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) < 2.0 ** -16 * float(want.detach())
    for n, q in model.named_parameters():
        off = (q.grad.double().cpu() - p[n].grad).norm() / p[n].grad.norm()
        assert off < 2.0 ** -13, (n, float(off))


def test_tokens_from_pools_follow_the_prompts():
    """A text fed as a prompt, or token by token from the pools: the same logits up to fp32 rounding of
    activations (2^-16 of their size after a few products)."""
    import recurrent_training as ex
    torch.backends.cuda.matmul.allow_tf32 = False
    model = ex.Model(seed=4)
    tokens, _, cu = ex.batch([12, 12, 12], seed=2)
    idx = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    whole = model.step(tokens, *model.pools(3), idx, cu)
    conv, state = model.pools(3)
    rows = tokens.view(3, 12)
    for t in range(12):
        got = model.step(rows[:, t].contiguous(), conv, state, idx)
        want = whole.view(3, 12, -1)[:, t]
        assert (got - want).abs().max() < 2.0 ** -16 * want.abs().max() * 16, t


def test_runs():
    import recurrent_training as ex
    model = ex.train(ex.Model(), steps=3)
    texts = ex.generate(model, [[1, 2, 3], [50]], tokens=4, temperature=0.7, top_k=10, top_p=0.9, min_p=0.01)
    assert len(texts) == 2 and all(len(t) == 4 and all(0 <= v < ex.VOCAB for v in t) for t in texts)
    again = ex.generate(model, [[1, 2, 3], [50]], tokens=4, temperature=0.7, top_k=10, top_p=0.9, min_p=0.01)
    assert texts == again
