"""A small hybrid recurrent model served with drafted tokens: a state space layer and a KDA layer, each
behind its short convolution, prompts first, then rounds of draft, verify and commit.

    python examples/hybrid_serving.py

The weights are random and the draft is a bigram table, so the text means nothing; what the example shows
is which call follows which and what each keeps:

  prompt   causal_conv -> ssm_scan          causal_conv -> chunk_prefill       (pools updated in place)
  round    causal_conv_draft -> ssm_decode_draft, causal_conv_draft -> decode_draft   (pools untouched,
           the state after every drafted token in a step cache)
           sample_probs -> the target's probabilities under temperature and filters
           verify_draft -> how many of the fed tokens stand, and the next one
           commit_draft, once a pool -> the state after the last token that stands
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_prefill_chunked_gb300 as kda  # noqa: E402

VOCAB, HID = 1000, 512
H, V, G, K = 8, 64, 1, 128        # state space layer: heads of 64 values, one group of 128 state channels
KH, KD = 4, 128                   # KDA layer: heads of 128 x 128
W = 4                             # taps of the convolutions
SSM_CH, KDA_CH = H * V + 2 * G * K, 3 * KH * KD


class Model:
    """Random weights and the two layers' pools for ``slots`` sequences (and the sentinel)."""

    def __init__(self, slots, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, std=None):
            return (torch.randn(*shape, generator=g, device="cuda") * (std or shape[-1] ** -0.5)).bfloat16()

        self.emb = w(VOCAB, HID, std=1.0)
        self.ssm_in, self.ssm_out = w(SSM_CH + H, HID), w(HID, H * V)
        self.kda_in, self.kda_out = w(KDA_CH + 2 * KH, HID), w(HID, KH * KD)
        self.head = w(VOCAB, HID, std=0.1)
        self.bigram = w(VOCAB, VOCAB, std=1.0)
        self.ssm_conv, self.kda_conv = w(SSM_CH, W, std=0.5), w(KDA_CH, W, std=0.5)
        self.a_log = torch.log(torch.rand(H, generator=g, device="cuda") * 15 + 1)
        self.dt_bias = torch.full((H,), -3.0, device="cuda")
        self.d = torch.ones(H, device="cuda")
        z = lambda *s, dt=torch.float32: torch.zeros(slots + 1, *s, device="cuda", dtype=dt)
        self.pools = dict(ssm_conv=z(W - 1, SSM_CH, dt=torch.bfloat16), ssm=z(H, K, V),
                          kda_conv=z(W - 1, KDA_CH, dt=torch.bfloat16), kda=z(KH, KD, KD))

    def caches(self, rows, steps):
        """Step caches: the pools' rows for every fed token of ``rows`` requests."""
        return {n: torch.zeros(rows, steps, *p.shape[1:], device="cuda", dtype=p.dtype)
                for n, p in self.pools.items()}

    def logits(self, tokens, cu, idx, caches=None):
        """Logits after each token; with ``caches`` the tokens are drafted ones of at most as many steps."""
        p, h = self.pools, self.emb[tokens.long()]
        steps = None if caches is None else caches["ssm"].shape[1]
        # state space layer: the convolution runs over x, B and C, slices of one projection
        proj = h @ self.ssm_in.T
        xbc, dt = proj[:, :SSM_CH], proj[:, SSM_CH:]
        if caches is None:
            xbc, _ = kda.causal_conv(xbc, self.ssm_conv, cu, activation="silu", state=p["ssm_conv"],
                                     state_indices=idx)
        else:
            xbc = kda.causal_conv_draft(xbc, self.ssm_conv, cu, p["ssm_conv"], idx, activation="silu",
                                        cache=caches["ssm_conv"], max_steps=steps)
        x, b, c = xbc.split([H * V, G * K, G * K], 1)
        args = (x.unflatten(1, (H, V)), dt, self.a_log, b.unflatten(1, (G, K)), c.unflatten(1, (G, K)), cu)
        if caches is None:
            y, _ = kda.ssm_scan(*args, D=self.d, dt_bias=self.dt_bias, state=p["ssm"], state_indices=idx)
        else:
            y = kda.ssm_decode_draft(*args, p["ssm"], idx, D=self.d, dt_bias=self.dt_bias,
                                     cache=caches["ssm"], max_steps=steps)
        h = h + y.flatten(1) @ self.ssm_out.T
        # KDA layer: the convolution runs over q, k and v; q and k are normalised in the kernel
        proj = h @ self.kda_in.T
        qkv, gate = proj[:, :KDA_CH], proj[:, KDA_CH:].float()
        if caches is None:
            qkv, _ = kda.causal_conv(qkv, self.kda_conv, cu, activation="silu", state=p["kda_conv"],
                                     state_indices=idx)
        else:
            qkv = kda.causal_conv_draft(qkv, self.kda_conv, cu, p["kda_conv"], idx, activation="silu",
                                        cache=caches["kda_conv"], max_steps=steps)
        q, k, v = (t.unflatten(1, (KH, KD)).contiguous() for t in qkv.split(KH * KD, 1))
        decay = -torch.nn.functional.softplus(gate[:, :KH]).contiguous()
        beta = torch.sigmoid(gate[:, KH:]).contiguous()
        if caches is None:
            o, _ = kda.chunk_prefill(q, k, v, decay, beta, cu, state=p["kda"], state_indices=idx,
                                     qk_l2norm=True)
        else:
            o = kda.decode_draft(q, k, v, decay, beta, cu, p["kda"], idx, cache=caches["kda"],
                                 max_steps=steps, qk_l2norm=True)
        h = h + o.flatten(1) @ self.kda_out.T
        return (h @ self.head.T).float()


def cu_of(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens).cumsum(0)
    return cu.cuda()


def serve(prompts, rounds=6, drafts=3, seed=1, temperature=1.0, top_k=None, top_p=None, min_p=None):
    """Prompts (lists of tokens) and what follows them: returns the model, the slots and the texts,
    whose last token has not been fed yet."""
    filters = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    n = len(prompts)
    m = Model(slots=n + 2)
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = torch.randperm(n + 2)[:n].to(torch.int32).cuda()
    exp = lambda *s: torch.empty(*s, device="cuda").exponential_(generator=g)

    flat = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device="cuda")
    cu = cu_of([len(p) for p in prompts])
    last = m.logits(flat, cu, idx)[cu[1:].long() - 1]
    fed = kda.sample(last, exp(n, VOCAB), **filters)
    texts = [list(p) + [int(t)] for p, t in zip(prompts, fed)]

    caches, steps = m.caches(n, drafts + 1), drafts + 1
    cu = cu_of([steps] * n)
    for _ in range(rounds):
        # the draft: tokens from the bigram table, one after another
        tokens, proposed = [fed], []
        for _ in range(drafts):
            logits = m.bigram[tokens[-1].long()]
            proposed.append(kda.sample_probs(logits, **filters))
            tokens.append(kda.sample(logits, exp(n, VOCAB), **filters))
        proposed.append(torch.zeros(n, VOCAB, device="cuda"))  # the last row is not read
        tokens = torch.stack(tokens, 1).flatten()
        q = torch.stack(proposed, 1).flatten(0, 1)
        # the target on all of them at once, then what stands of them
        p = kda.sample_probs(m.logits(tokens, cu, idx, caches), **filters)
        u = torch.rand(n * steps, generator=g, device="cuda")
        kept, fed = kda.verify_draft(tokens, p, q, u, exp(n, VOCAB), cu)
        for name, pool in m.pools.items():
            kda.commit_draft(caches[name], kept, pool, idx)
        for text, row, k, t in zip(texts, tokens.view(n, steps).tolist(), kept.tolist(), fed.tolist()):
            text += row[1:k] + [t]
    return m, idx, texts


def main():
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(VOCAB, (int(n),), generator=g).tolist() for n in (5, 70, 200, 1)]
    m, idx, texts = serve(prompts)
    for p, t in zip(prompts, texts):
        print(f"prompt of {len(p)} tokens, {len(t) - len(p)} generated: {t[len(p):]}")
    # the committed pools against the same texts fed as prompts from nothing
    again = Model(slots=idx.numel() + 2)
    again.logits(torch.tensor([t for x in texts for t in x[:-1]], dtype=torch.int32, device="cuda"),
                 cu_of([len(x) - 1 for x in texts]), idx)
    worst = 0.0
    for name, pool in m.pools.items():
        a, b = pool[idx.long()].float(), again.pools[name][idx.long()].float()
        e = float((a - b).norm() / b.norm())
        worst = max(worst, e)
        print(f"pool {name:9s} against the texts as prompts: relative difference {e:.1e}")
    return worst


if __name__ == "__main__":
    main()
