"""A small recurrent model trained, then served: a short convolution and a gated linear recurrence over packed
sequences of different lengths, forward and backward, then prompts and tokens from pools of states.

    python examples/recurrent_training.py

The sequences count up in steps of their own, modulo the vocabulary.  The library's calls are plain functions;
``Conv`` and ``Gated`` make them nodes of PyTorch's autograd, with each sequence's state as a tensor that
gradients pass through, too.

  training  causal_conv, gated_scan (output_carries=True)  ->  causal_conv_backward, gated_scan_backward
  prompt    causal_conv, gated_scan on pools                     (updated in place)
  token     causal_conv_decode, gated_decode, sample
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_prefill_chunked_gb300 as kda  # noqa: E402

VOCAB, HID, W = 97, 256, 4


class Conv(torch.autograd.Function):
    """(x [T, Ch], weight, bias, state [N, W-1, Ch]) -> (y, final state), with SiLU."""

    @staticmethod
    def forward(ctx, x, weight, bias, state, cu):
        ctx.save_for_backward(x, weight, bias, state, cu)
        return kda.causal_conv(x, weight, cu, bias=bias, activation="silu", state=state)

    @staticmethod
    def backward(ctx, dy, dfinal):
        x, weight, bias, state, cu = ctx.saved_tensors
        dx, dw, db, dstate = kda.causal_conv_backward(dy.contiguous(), x, weight, cu, bias=bias, activation="silu",
                                                      state=state, dfinal=dfinal.contiguous())
        return dx, dw.to(weight.dtype), db.to(bias.dtype), dstate, None


class Gated(torch.autograd.Function):
    """(x, r, i [T, Ch], A_log [Ch], state [N, Ch]) -> (y, final state)."""

    @staticmethod
    def forward(ctx, x, r, i, A_log, state, cu):
        y, final, carries = kda.gated_scan(x, r, A_log, cu, i=i, state=state, output_carries=True)
        ctx.save_for_backward(x, r, i, A_log, state, cu, carries)
        return y, final

    @staticmethod
    def backward(ctx, dy, dfinal):
        x, r, i, A_log, state, cu, carries = ctx.saved_tensors
        dx, dr, di, da, dstate = kda.gated_scan_backward(dy.contiguous(), x, r, A_log, cu, carries, i=i, state=state,
                                                         dfinal=dfinal.contiguous())
        return dx, dr, di, da, dstate, None


class Model(torch.nn.Module):
    def __init__(self, seed=0, dtype=torch.float32):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        w = lambda *s, std=None: torch.nn.Parameter(
            (torch.randn(*s, generator=g) * (std or s[-1] ** -0.5)).to(dtype).cuda())
        self.emb, self.head = w(VOCAB, HID, std=1.0), w(VOCAB, HID)
        self.conv_w, self.conv_b = w(HID, W, std=0.5), w(HID, std=0.1)
        self.gates, self.out = w(2 * HID, HID), w(HID, HID)
        decay = -8.0 * torch.log(0.9 + 0.099 * torch.rand(HID, generator=g))
        self.A_log = torch.nn.Parameter(torch.log(decay).cuda())
        self.conv_h0, self.h0 = w(W - 1, HID, std=0.1), torch.nn.Parameter((torch.randn(HID, generator=g) * 0.1).cuda())

    def forward(self, tokens, cu):
        """Logits of packed sequences; every sequence starts from the model's own states."""
        n = cu.numel() - 1
        x = self.emb[tokens.long()]
        u, _ = Conv.apply(x, self.conv_w, self.conv_b, self.conv_h0.expand(n, -1, -1).contiguous(), cu)
        r, i = (u @ self.gates.T).split(HID, 1)
        y, _ = Gated.apply(u, r, i, self.A_log, self.h0.expand(n, -1).contiguous(), cu)
        return (x + y @ self.out.T) @ self.head.T

    def pools(self, slots):
        """The states of ``slots`` sequences (and the sentinel), as they begin."""
        return (self.conv_h0.detach().expand(slots + 1, -1, -1).contiguous(),
                self.h0.detach().expand(slots + 1, -1).contiguous())

    @torch.no_grad()
    def step(self, tokens, conv, state, idx, cu=None):
        """Logits from pools: of one token a row, or of packed prompts."""
        x = self.emb[tokens.long()]
        if cu is None:
            u = kda.causal_conv_decode(x, self.conv_w, conv, idx, bias=self.conv_b, activation="silu")
            r, i = (u @ self.gates.T).split(HID, 1)
            y = kda.gated_decode(u, r, self.A_log, state, idx, i=i)
        else:
            u, _ = kda.causal_conv(x, self.conv_w, cu, bias=self.conv_b, activation="silu", state=conv,
                                   state_indices=idx)
            r, i = (u @ self.gates.T).split(HID, 1)
            y, _ = kda.gated_scan(u, r, self.A_log, cu, i=i, state=state, state_indices=idx)
        return (x + y @ self.out.T) @ self.head.T


def batch(lens, seed):
    """Counting sequences of the given lengths: tokens, the tokens after them, cu_seqlens."""
    g = torch.Generator().manual_seed(seed)
    seqs = [(int(torch.randint(VOCAB, (1,), generator=g)) + int(torch.randint(1, 5, (1,), generator=g))
             * torch.arange(n + 1)) % VOCAB for n in lens]
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens).cumsum(0)
    return (torch.cat([s[:-1] for s in seqs]).to(torch.int32).cuda(), torch.cat([s[1:] for s in seqs]).cuda(),
            cu.cuda())


def train(model, steps=60, lr=3e-3):
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    for k in range(steps):
        tokens, after, cu = batch([50, 0, 7, 130, 1, 64], seed=k)
        loss = torch.nn.functional.cross_entropy(model(tokens, cu).float(), after)
        opt.zero_grad()
        loss.backward()
        opt.step()
        if k % 20 == 0 or k == steps - 1:
            print(f"step {k:3d} loss {float(loss.detach()):.3f}")
    return model


def generate(model, prompts, tokens=8, seed=0, **filters):
    """Tokens after the prompts (lists), drawn from pools of states."""
    n = len(prompts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    conv, state = model.pools(n)
    idx = torch.arange(n, dtype=torch.int32, device="cuda")
    cu = torch.zeros(n + 1, dtype=torch.int32)
    cu[1:] = torch.tensor([len(p) for p in prompts]).cumsum(0)
    cu = cu.cuda()
    flat = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device="cuda")
    logits = model.step(flat, conv, state, idx, cu)[cu[1:].long() - 1]
    texts = []
    for _ in range(tokens):
        noise = torch.empty(n, VOCAB, device="cuda").exponential_(generator=g)
        fed = kda.sample(logits, noise, **filters)
        texts.append(fed)
        logits = model.step(fed, conv, state, idx)
    return torch.stack(texts, 1).tolist()


def main():
    model = train(Model())
    prompts = [list(range(3, 40, 2)), list(range(10, 20)), [5, 9, 13, 17, 21]]
    for p, t in zip(prompts, generate(model, prompts, temperature=0.5, top_k=5, top_p=0.9)):
        print(f"{p} -> {t}")


if __name__ == "__main__":
    main()
