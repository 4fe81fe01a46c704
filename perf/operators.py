"""The recurrent-layer operators that a host of the KDA kernels runs next to them, as cases with
inputs, a plain form, a 64-bit form and the work that no form can do without.

Four operators in their serving forms:

  conv_prompt, conv_token    short causal depthwise convolution (with SiLU) of packed prompts, and of
                             one token (or a few drafted ones) a request, on a pool of its last inputs
  scan_prompt, scan_token    selective state space scan of packed prompts, and of one token (or a few
                             drafted ones) a request, on a pool of states
  verify                     drafted tokens against the target's probabilities, from given random numbers
  commit                     the state after the accepted tokens, from the draft steps' states into a pool

``run`` computes a case in elementary torch operations where ``own`` is false, and by the
framework's own calls where it is true.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # The short convolution of the q, k and v channels (3 x 32 heads x 128) before the prefill
        # of the throughput workload: 32768 tokens as 16 sequences of log-uniform lengths.
        dict(name="conv prompt 32768x12288", op="conv_prompt", tokens=32768, seqs=16, lens="log",
             lens_seed=0, channels=12288, width=4, silu=True, bias=False, dtype="bf16", pool=True),
        # An odd channel count, a 3-tap filter with a bias and no activation, in fp32, over many
        # short sequences, some of them empty: rows that no vector access fits.
        dict(name="conv prompt ragged fp32", op="conv_prompt", tokens=2741, seqs=37, lens="empty",
             lens_seed=3, channels=1003, width=3, silu=False, bias=True, dtype="fp32", pool=False),
        # One decode step of 64 requests through the same convolution: a latency-bound call.
        dict(name="conv token 64x12288", op="conv_token", rows=64, steps=1, channels=12288, width=4,
             silu=True, bias=True, dtype="bf16", slots=80),
        # The throughput workload's lengths and heads (32 of 128 x 128), 8 groups, fp32 pool.
        dict(name="scan prompt 32768 16 seqs", op="scan_prompt", tokens=32768, seqs=16, lens="log",
             lens_seed=0, heads=32, groups=8, K=128, V=128, dtype="bf16", state="fp32", pool=True),
        # One long prompt alone, 64 heads of 64 in one group: few sequences, so the time axis has to
        # be split to fill the GPU.
        dict(name="scan prompt 8192 1 seq", op="scan_prompt", tokens=8192, seqs=1, lens="log",
             lens_seed=0, heads=64, groups=1, K=128, V=64, dtype="bf16", state="fp32", pool=False),
        # Many short prompts in fp32 with 64-wide heads, some empty: the odd end of the range.
        dict(name="scan prompt ragged fp32", op="scan_prompt", tokens=2209, seqs=24, lens="empty",
             lens_seed=5, heads=6, groups=2, K=64, V=64, dtype="fp32", state="fp32", pool=False),
        # A large decode batch: the states of 1024 requests streamed once (2 GiB in, 2 GiB out).
        dict(name="scan token 1024 rows", op="scan_token", rows=1024, steps=1, heads=32, groups=8,
             K=128, V=128, dtype="bf16", state="fp32", slots=1040),
        # A few requests with four drafted tokens each: every step's state is kept.
        dict(name="scan draft 8x4", op="scan_token", rows=8, steps=4, heads=32, groups=4, K=128, V=64,
             dtype="bf16", state="fp32", slots=16),
        # Verification for a serving batch with a large vocabulary.
        dict(name="verify 64x4 131072", op="verify", rows=64, drafts=4, vocab=131072),
        # One request with an odd vocabulary: the smallest call.
        dict(name="verify 1x3 32003", op="verify", rows=1, drafts=3, vocab=32003),
        # The accepted states of 128 requests (32 heads of 128 x 128, fp32) into the pool.
        dict(name="commit 128 states", op="commit", rows=128, steps=5, heads=32, K=128, V=128,
             dtype="fp32", slots=140),
        # The same for the convolution's few inputs a request.
        dict(name="commit 8 conv inputs", op="commit", rows=8, steps=4, heads=1, K=3, V=4096, dtype="bf16",
             slots=20),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_prompt", "conv_token", "scan_prompt", "scan_prompt", "scan_token",
                     "verify", "commit"])
    if op == "conv_prompt":
        tokens = _log(rng, 1, 32768)
        ch = _log(rng, 16, 12288)
        if rng.random() < 0.7:
            ch = max(8, ch // 8 * 8)
        return dict(op=op, tokens=tokens, seqs=min(tokens, _log(rng, 1, 128)),
                    lens=rng.choice(["log", "empty"]), lens_seed=rng.randrange(1 << 20), channels=ch,
                    width=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7, bias=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), pool=rng.random() < 0.5)
    if op == "conv_token":
        rows = _log(rng, 1, 2048)
        ch = _log(rng, 16, 12288)
        if rng.random() < 0.7:
            ch = max(8, ch // 8 * 8)
        return dict(op=op, rows=rows, steps=rng.choice([1, 1, 2, 3, 5]), channels=ch,
                    width=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7, bias=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), slots=rows + rng.randrange(1, 40))
    if op == "scan_prompt":
        bf16 = rng.random() < 0.75
        K, V = rng.choice([(128, 64), (128, 128), (128, 64), (64, 64), (64, 128)])
        heads = rng.choice([3, 8, 16, 24, 32] + ([48, 64] if V == 64 else []))
        tokens = _log(rng, 1, 32768 if bf16 else 8192)
        return dict(op=op, tokens=tokens, seqs=min(tokens, _log(rng, 1, 64)),
                    lens=rng.choice(["log", "log", "empty"]), lens_seed=rng.randrange(1 << 20),
                    heads=heads, groups=rng.choice([g for g in (1, 2, 3, 8) if heads % g == 0]), K=K,
                    V=V, dtype="bf16" if bf16 else "fp32",
                    state=rng.choice(["fp32", "fp32", "bf16"]) if bf16 else "fp32",
                    pool=rng.random() < 0.5)
    if op == "scan_token":
        rows, steps = _log(rng, 1, 768), rng.choice([1, 1, 2, 3, 5])
        heads = rng.choice([3, 8, 16, 32])
        return dict(op=op, rows=rows if steps == 1 else max(1, rows // 6), steps=steps, heads=heads,
                    groups=rng.choice([g for g in (1, 2, 3, 8) if heads % g == 0]),
                    K=rng.choice([64, 128, 128]), V=rng.choice([64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    state=rng.choice(["fp32", "fp32", "bf16"]), slots=rows + rng.randrange(1, 20))
    if op == "verify":
        vocab = _log(rng, 500, 200000)
        rows = max(1, min(_log(rng, 1, 256), 64 * 131072 // vocab))
        return dict(op=op, rows=rows, drafts=rng.randrange(1, 6), vocab=vocab)
    if rng.random() < 0.5:
        row = dict(heads=rng.choice([8, 16, 32]), K=rng.choice([64, 128]), V=rng.choice([64, 128]))
        rows = _log(rng, 1, 128)
    else:
        row, rows = dict(heads=1, K=rng.randrange(1, 4), V=_log(rng, 16, 12288)), _log(rng, 1, 512)
    return dict(op=op, rows=rows, steps=rng.randrange(1, 6), **row,
                dtype=rng.choice(["fp32", "bf16"]), slots=rows + rng.randrange(1, 20))


def lengths(case):
    """Sequence lengths of a prompt case: log-uniform shares of its tokens; "empty": some are 0."""
    r = random.Random(case["lens_seed"])
    n, total = case["seqs"], case["tokens"]
    share = [math.exp(r.uniform(math.log(64), math.log(8192))) for _ in range(n)]
    if case["lens"] == "empty":
        share = [0.0 if i % 5 == 2 else s for i, s in enumerate(share)]
    top = sum(share)
    lens = [int(s * total / top) for s in share]
    lens[share.index(max(share))] += total - sum(lens)
    return lens


def steps_of(case):
    """Tokens of each request of a draft case: up to ``steps``, a few requests with fewer."""
    return [case["steps"] - (i % 3 if case["steps"] > 2 else 0) for i in range(case["rows"])]


def _cu(lens, device):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return torch.tensor(cu, dtype=torch.int32, device=device)


# ------------------------------------------------------------------------------ the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def slots(rows, count, pad):
        """Distinct slots of the pool; one row of a larger batch is padding (-1: the last slot)."""
        idx = torch.randperm(count - 1, generator=g, device=dev)[:rows].to(torch.int32)
        if pad and rows > 1:
            idx[rows // 2] = -1
        return idx

    op = case["op"]
    st = dict(case=case, op=op)
    if op in ("conv_prompt", "conv_token"):
        dt, ch, w = DT[case["dtype"]], case["channels"], case["width"]
        lens = lengths(case) if op == "conv_prompt" else steps_of(case)
        t, n = sum(lens), len(lens)
        st.update(cu=_cu(lens, dev), x=normal(t, ch).to(dt), weight=normal(ch, w, std=0.5).to(dt),
                  bias=normal(ch, std=0.1).to(dt) if case["bias"] else None,
                  act="silu" if case["silu"] else None)
        if op == "conv_prompt" and not case["pool"]:
            st.update(state=normal(n, w - 1, ch).to(dt), idx=None)
        else:
            count = case.get("slots", n + 3)
            st.update(state=normal(count, w - 1, ch).to(dt), idx=slots(n, count, True))
        if op == "conv_token" and case["steps"] > 1:
            st.update(cache=torch.zeros(n, case["steps"], w - 1, ch, dtype=dt, device=dev))
    elif op in ("scan_prompt", "scan_token"):
        dt, sd = DT[case["dtype"]], DT[case["state"]]
        h, grp, k, v = case["heads"], case["groups"], case["K"], case["V"]
        lens = lengths(case) if op == "scan_prompt" else steps_of(case)
        t, n = sum(lens), len(lens)
        # x, B and C are slices of the convolution's output, as a layer has them
        xbc = torch.nn.functional.silu(normal(t, h * v + 2 * grp * k)).to(dt)
        step = torch.exp(uniform(h) * math.log(100.0) + math.log(1e-3))
        st.update(cu=_cu(lens, dev), x=xbc[:, :h * v].unflatten(1, (h, v)),
                  B=xbc[:, h * v:h * v + grp * k].unflatten(1, (grp, k)),
                  C=xbc[:, h * v + grp * k:].unflatten(1, (grp, k)), dt=normal(t, h).to(dt),
                  A_log=torch.log(uniform(h) * 15.0 + 1.0), dt_bias=torch.log(torch.expm1(step)),
                  D=normal(h, std=0.2) + 1.0)
        if op == "scan_prompt" and not case["pool"]:
            st.update(state=normal(n, h, k, v, std=0.1).to(sd), idx=None)
        else:
            count = case.get("slots", n + 3)
            pool = torch.empty(count, h, k, v, dtype=sd, device=dev)
            for i in range(0, count, 64):
                pool[i:i + 64] = normal(min(64, count - i), h, k, v, std=0.1).to(sd)
            st.update(state=pool, idx=slots(n, count, True))
        if op == "scan_token" and case["steps"] > 1:
            st.update(cache=torch.zeros(n, case["steps"], h, k, v, dtype=sd, device=dev))
    elif op == "verify":
        # a request is fed its last token and the drafted ones; row t of the probabilities follows
        # token t.  The draft's distribution is near the target's, its tokens are drawn from it.
        n, vocab = case["rows"], case["vocab"]
        lens = [case["drafts"] + 1 - (i % 4 == 3) for i in range(n)]
        t = sum(lens)
        logits = normal(t, vocab, std=2.5)
        near = logits + normal(t, vocab, std=0.4)
        e = torch.empty(t, vocab, device=dev).exponential_(generator=g)
        nxt = torch.argmax(near - torch.log(e.clamp_min(1e-30)), dim=1)
        st.update(cu=_cu(lens, dev), target=torch.softmax(logits, 1), draft=torch.softmax(near, 1),
                  tokens=torch.roll(nxt, 1).to(torch.int32), u=uniform(t),
                  noise=torch.empty(n, vocab, device=dev).exponential_(generator=g).clamp_min(1e-30))
    else:
        dt, row = DT[case["dtype"]], (case["heads"], case["K"], case["V"])
        n, s = case["rows"], case["steps"]
        cache = torch.empty(n, s, *row, dtype=dt, device=dev)
        for i in range(0, n, 32):
            cache[i:i + 32] = normal(min(32, n - i), s, *row).to(dt)
        st.update(cache=cache, pool=normal(case["slots"], *row).to(dt), idx=slots(n, case["slots"], True),
                  accepted=torch.randint(0, s + 1, (n,), generator=g, device=dev, dtype=torch.int32))
    return st


# ------------------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import linear_attention_prefill_chunked_gb300 as kda
    op = s["op"]
    if op == "conv_prompt":
        y, final = kda.causal_conv(s["x"], s["weight"], s["cu"], bias=s["bias"], activation=s["act"],
                                   state=s["state"], state_indices=s["idx"])
        return {"y": y, "state": final}
    if op == "conv_token":
        if "cache" in s:
            y = kda.causal_conv_draft(s["x"], s["weight"], s["cu"], s["state"], s["idx"], bias=s["bias"],
                                      activation=s["act"], cache=s["cache"],
                                      max_steps=s["cache"].shape[1])
            return {"y": y, "cache": s["cache"]}
        y = kda.causal_conv_decode(s["x"], s["weight"], s["state"], s["idx"], bias=s["bias"],
                                   activation=s["act"])
        return {"y": y, "state": s["state"]}
    if op == "scan_prompt":
        y, final = kda.ssm_scan(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["cu"], D=s["D"],
                                dt_bias=s["dt_bias"], state=s["state"], state_indices=s["idx"])
        return {"y": y, "state": final}
    if op == "scan_token":
        if "cache" in s:
            y = kda.ssm_decode_draft(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["cu"], s["state"],
                                     s["idx"], D=s["D"], dt_bias=s["dt_bias"], cache=s["cache"],
                                     max_steps=s["cache"].shape[1])
            return {"y": y, "cache": s["cache"]}
        y = kda.ssm_decode(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["state"], s["idx"], D=s["D"],
                           dt_bias=s["dt_bias"])
        return {"y": y, "state": s["state"]}
    if op == "verify":
        kept, token = kda.verify_draft(s["tokens"], s["target"], s["draft"], s["u"], s["noise"], s["cu"])
        return {"kept": kept, "token": token}
    return {"pool": kda.commit_draft(s["cache"], s["accepted"], s["pool"], s["idx"])}


def _run_plain(s):
    op = s["op"]
    if op in ("conv_prompt", "conv_token"):
        return _plain_conv(s)
    if op == "scan_prompt":
        return _plain_scan(s)
    if op == "scan_token":
        return _plain_scan_token(s)
    if op == "verify":
        return _plain_verify(s)
    n = s["accepted"].shape[0]
    slot = _slot(s["idx"], s["pool"])
    kept = s["accepted"].long()
    row = s["cache"][torch.arange(n, device=kept.device), (kept - 1).clamp_min(0)]
    keep = (kept > 0).view(n, *[1] * (row.dim() - 1))
    s["pool"][slot] = torch.where(keep, row, s["pool"][slot])
    return {"pool": s["pool"]}


def _slot(idx, pool):
    return torch.where(idx < 0, pool.shape[0] - 1, idx).long()


def _plain_conv(s):
    """y_t = act(bias + sum_i w_i x_{t-(W-1)+i}), the inputs before a sequence from its state."""
    x, w = s["x"], s["weight"].float()
    t, width = x.shape[0], w.shape[1]
    cu = s["cu"].long()
    n = cu.shape[0] - 1
    seq = torch.repeat_interleave(torch.arange(n, device=x.device), cu[1:] - cu[:-1], output_size=t)
    pos = torch.arange(t, device=x.device) - cu[seq]
    h0 = s["state"] if s["idx"] is None else s["state"][_slot(s["idx"], s["state"])]
    both = torch.cat([h0.reshape(n * (width - 1), -1), x]).float()

    def source(q, back, first):
        """Row of ``both`` that lies ``back`` inputs before position ``pos`` of sequence ``q``."""
        at, start = first
        return torch.where(at >= back, n * (width - 1) + start + at - back,
                           q * (width - 1) + (width - 1) + at - back)

    first = (pos, cu[seq])
    y = sum(both[source(seq, width - 1 - i, first)] * w[:, i] for i in range(width))
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["act"] == "silu":
        y = y * torch.sigmoid(y)
    y = y.to(x.dtype)
    back = torch.arange(width - 2, -1, -1, device=x.device)
    if "cache" in s:  # the inputs kept after each draft step
        steps = both[source(seq[:, None], back[None], (pos[:, None], cu[seq][:, None]))].to(x.dtype)
        s["cache"][seq, pos] = steps
        return {"y": y, "cache": s["cache"]}
    each = torch.arange(n, device=x.device)[:, None]
    last = (cu[1:] - cu[:-1] - 1)[:, None]
    final = both[source(each, back[None], (last, cu[:-1][:, None]))].to(x.dtype)
    if s["idx"] is None:
        return {"y": y, "state": final}
    s["state"][_slot(s["idx"], s["state"])] = final
    return {"y": y, "state": s["state"]}


def _steps(s):
    """Step sizes softplus(dt + bias) and log-decays -exp(A_log) * step, both [T, H] in 32 bits."""
    z = s["dt"].float() + s["dt_bias"]
    step = torch.clamp_min(z, 0.0) + torch.log1p(torch.exp(-torch.abs(z)))
    return step, -torch.exp(s["A_log"]) * step


def _plain_scan(s):
    """Chunked form: within a chunk by a decayed score matrix, between chunks by a decay matrix."""
    x, L = s["x"], CHUNK
    t, h, v = x.shape
    grp, k = s["B"].shape[1:]
    dev = x.device
    cu = s["cu"].long()
    n = cu.shape[0] - 1
    h0 = (s["state"] if s["idx"] is None else s["state"][_slot(s["idx"], s["state"])]).float()
    nch = (cu[1:] - cu[:-1] + L - 1) // L
    end = torch.cumsum(nch, 0)
    chunk = torch.arange(t // L + n, device=dev)
    seq = torch.searchsorted(end, chunk, right=True)
    real = seq < n
    seq = seq.clamp_max(n - 1)
    tok = (cu[seq] + (chunk - (end - nch)[seq]) * L)[:, None] + torch.arange(L, device=dev)
    ok = real[:, None] & (tok < cu[seq + 1][:, None])
    tok = tok.clamp(0, t - 1)
    step, g = _steps(s)
    step, g = (torch.where(ok[..., None], a[tok], 0.0).permute(0, 2, 1) for a in (step, g))  # [n, h, L]
    xc = torch.where(ok[..., None, None], x[tok].float(), 0.0)
    bc, cc = (torch.where(ok[..., None, None], a[tok].float(), 0.0) for a in (s["B"], s["C"]))
    # decay between two tokens of a chunk: the sum of the log-decays after s up to t
    after = torch.ones(L, L, dtype=torch.bool, device=dev).tril(-1)
    span = torch.cumsum(torch.where(after, g[..., :, None], 0.0), 2)
    decay = torch.where(after | torch.eye(L, dtype=torch.bool, device=dev), torch.exp(span), 0.0)
    score = torch.einsum("nlgk,nsgk->ngls", cc, bc).repeat_interleave(h // grp, 1)
    score = score * decay * step[:, :, None, :]
    y = torch.einsum("nhls,nshv->nlhv", score, xc)
    # the state that each chunk adds, and the state before each chunk
    bh = bc.repeat_interleave(h // grp, 2)
    weight = (decay[:, :, -1] * step).permute(0, 2, 1)[..., None]
    add = torch.einsum("nshk,nshv->nhkv", bh * weight, xc)
    total = g.sum(2)                                                   # [chunks, h]
    m = chunk.shape[0]
    tri = torch.ones(m, m, dtype=torch.bool, device=dev).tril(-1)      # [later, earlier]
    run_ = torch.cumsum(torch.where(tri, total.T[:, :, None], 0.0), 1)  # decay after chunk j up to i
    same = (seq[:, None] == seq[None, :]) & real[:, None] & real[None, :]
    till = torch.where(same & (tri | torch.eye(m, dtype=torch.bool, device=dev)), torch.exp(run_), 0.0)
    head = torch.zeros(m, dtype=torch.bool, device=dev)
    start = (end - nch).clamp_max(m - 1)
    first = (chunk == start[seq]) & real
    # the initial state counts as an addition to a sequence's first chunk, decayed over it
    add = add + torch.where(first[:, None, None, None], torch.exp(total)[..., None, None] * h0[seq], 0.0)
    post = torch.einsum("hij,jhkv->ihkv", till, add)                   # state after each chunk
    before = torch.where(first[:, None, None, None], h0[seq], torch.roll(post, 1, 0))
    since = torch.exp(torch.cumsum(g, 2)).permute(0, 2, 1)[..., None]
    ch = cc.repeat_interleave(h // grp, 2)
    y = y + torch.einsum("nlhk,nhkv->nlhv", ch * since, before)
    y = y + s["D"][:, None] * xc
    out = torch.empty(t + 1, h, v, device=dev)
    out[torch.where(ok, tok, t)] = y
    final = torch.where((nch > 0)[:, None, None, None], post[(end - 1).clamp_min(0)], h0)
    y, final = out[:t].to(x.dtype), final.to(s["state"].dtype)
    if s["idx"] is None:
        return {"y": y, "state": final}
    s["state"][_slot(s["idx"], s["state"])] = final
    return {"y": y, "state": s["state"]}


def _plain_scan_token(s):
    x = s["x"]
    t, h, v = x.shape
    grp = s["B"].shape[1]
    cu = s["cu"].long()
    n = cu.shape[0] - 1
    step, g = _steps(s)
    bh, ch = (a.float().repeat_interleave(h // grp, 1) for a in (s["B"], s["C"]))
    xf = x.float()
    h0 = s["state"][_slot(s["idx"], s["state"])].float()
    if "cache" not in s:
        new = torch.exp(g)[..., None, None] * h0 + (step[..., None] * bh)[..., None] * xf[:, :, None]
        y = (new * ch[..., None]).sum(2) + s["D"][:, None] * xf
        s["state"][_slot(s["idx"], s["state"])] = new.to(s["state"].dtype)
        return {"y": y.to(x.dtype), "state": s["state"]}
    # the state after step j of a request: its start and the additions of the steps up to j, decayed
    m = s["cache"].shape[1]
    j = torch.arange(m, device=x.device)
    ok = j[None] < (cu[1:] - cu[:-1])[:, None]
    tok = (cu[:-1, None] + j).clamp_max(t - 1)
    gj = torch.where(ok[..., None], g[tok], 0.0).permute(0, 2, 1)
    after = torch.ones(m, m, dtype=torch.bool, device=x.device).tril(-1)
    span = torch.cumsum(torch.where(after, gj[..., :, None], 0.0), 2)
    decay = torch.where(after | torch.eye(m, dtype=torch.bool, device=x.device), torch.exp(span), 0.0)
    add = (step[..., None] * bh)[..., None] * xf[:, :, None]
    add = torch.where(ok[..., None, None, None], add[tok], 0.0)         # [n, m, h, k, v]
    st = torch.einsum("nhji,nihkv->njhkv", decay, add)
    st = st + torch.exp(torch.cumsum(gj, 2)).permute(0, 2, 1)[..., None, None] * h0[:, None]
    seq = torch.repeat_interleave(torch.arange(n, device=x.device), cu[1:] - cu[:-1], output_size=t)
    pos = torch.arange(t, device=x.device) - cu[seq]
    mine = st[seq, pos]
    y = (mine * ch[..., None]).sum(2) + s["D"][:, None] * xf
    s["cache"][seq, pos] = mine.to(s["cache"].dtype)
    return {"y": y.to(x.dtype), "cache": s["cache"]}


def _plain_verify(s):
    """Draft j + 1 is kept while u q(d) < p(d); then one token by an exponential race: from max(p - q, 0)
    after a refusal, from p if no draft was refused (or nothing is left of the difference)."""
    p, q, cu = s["target"], s["draft"], s["cu"].long()
    t, vocab = p.shape
    n = cu.shape[0] - 1
    dev = p.device
    lens = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(n, device=dev), lens, output_size=t)
    at = torch.arange(t, device=dev)
    nxt = s["tokens"].long().roll(-1)[:, None]
    good = s["u"] * q.gather(1, nxt)[:, 0] < p.gather(1, nxt)[:, 0]
    stop = ~good | (at == cu[seq + 1] - 1)
    kept = torch.full((n,), t, dtype=torch.long, device=dev)
    kept = kept.scatter_reduce(0, seq, torch.where(stop, at, t), "amin")
    last = kept.clamp_max(t - 1)
    refused = (kept < cu[1:] - 1)[:, None]
    pr = p[last]
    diff = torch.clamp_min(pr - q[last], 0.0)
    r = torch.where(refused & (diff > 0).any(1, keepdim=True), diff, pr)
    score = torch.where(r > 0, r / s["noise"], -1.0)
    best = score.max(1, keepdim=True).values
    token = torch.where(score == best, torch.arange(vocab, device=dev), vocab).min(1).values
    token = torch.where(best[:, 0] < 0, -1, token)
    return {"kept": (kept - cu[:-1] + 1).to(torch.int32), "token": token.to(torch.int32)}


# ------------------------------------------------------------------------------ the work

def work(case):
    """Bytes of each input read once and each output written once, and the operations of the formulas."""
    size = {"bf16": 2, "fp32": 4}
    op = case["op"]
    if op in ("conv_prompt", "conv_token"):
        e, ch, w = size[case["dtype"]], case["channels"], case["width"]
        lens = lengths(case) if op == "conv_prompt" else steps_of(case)
        t, n = sum(lens), len(lens)
        states = n * (w - 1) * ch * e
        new = t * (w - 1) * ch * e if op == "conv_token" and case["steps"] > 1 else states
        return {"bytes": 2 * t * ch * e + states + new + ch * (w + 1) * e, "flops": 2 * t * ch * (w + 2)}
    if op in ("scan_prompt", "scan_token"):
        e, se = size[case["dtype"]], size[case["state"]]
        h, grp, k, v = case["heads"], case["groups"], case["K"], case["V"]
        lens = lengths(case) if op == "scan_prompt" else steps_of(case)
        t, n = sum(lens), len(lens)
        states = n * h * k * v * se
        new = t * h * k * v * se if op == "scan_token" and case["steps"] > 1 else states
        return {"bytes": t * e * (2 * h * v + 2 * grp * k + h) + states + new + 12 * h,
                "flops": t * h * (5 * k * v + 2 * v)}
    if op == "verify":
        # one row of the target's probabilities and the noise a request, and the draft's where refused
        lens = [case["drafts"] + 1 - (i % 4 == 3) for i in range(case["rows"])]
        rows = case["rows"]
        return {"bytes": rows * case["vocab"] * (4 + 4 + 2) + sum(lens) * 16 + 8 * rows,
                "flops": 3 * rows * case["vocab"]}
    row = case["heads"] * case["K"] * case["V"] * size[case["dtype"]]
    share = case["steps"] / (case["steps"] + 1)
    return {"bytes": 2 * row * case["rows"] * share, "flops": 0}


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions token by token in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "conv_prompt" or op == "conv_token":
        return _exact_conv(s, case)
    if op in ("scan_prompt", "scan_token"):
        return _exact_scan(s, case)
    if op == "verify":
        return _exact_verify(s)
    pool = s["pool"].double()
    for i, (j, a) in enumerate(zip(s["idx"].tolist(), s["accepted"].tolist())):
        if a > 0:
            pool[j] = s["cache"][i, a - 1].double()  # -1 is the last row
    return {"pool": pool}


def _exact_conv(s, case):
    cu = s["cu"].tolist()
    w, x = s["weight"].double(), s["x"].double()
    width = w.shape[1]
    state = s["state"].double()
    final = state.clone()
    y = torch.empty_like(x)
    cache = s["cache"].double() if "cache" in s else None
    idx = list(range(len(cu) - 1)) if s["idx"] is None else s["idx"].tolist()
    for i, slot in enumerate(idx):
        a, b = cu[i], cu[i + 1]
        ext = torch.cat([state[slot], x[a:b]])
        y[a:b] = (ext.unfold(0, width, 1)[:b - a] * w).sum(-1) if b > a else 0.0
        final[slot] = ext[b - a:]
        if cache is not None:
            for j in range(b - a):
                cache[i, j] = ext[j + 1:j + width]
    if s["bias"] is not None:
        y += s["bias"].double()
    if s["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    return {"y": y, "cache": cache} if cache is not None else {"y": y, "state": final}


def _exact_scan(s, case):
    x = s["x"].double()
    t, h, v = x.shape
    rep = h // s["B"].shape[1]
    cu = s["cu"].long()
    n = cu.shape[0] - 1
    lens = cu[1:] - cu[:-1]
    longest = int(lens.max())
    z = s["dt"].double() + s["dt_bias"].double()
    step = torch.logaddexp(z, torch.zeros_like(z))
    keep = torch.exp(-torch.exp(s["A_log"].double()) * step)
    slot = torch.arange(n, device=x.device) if s["idx"] is None else _slot(s["idx"], s["state"])
    S = s["state"][slot].double()
    if longest * (S.numel() * 48 / 4e12 + 1e-4) > 15:
        return None
    y = torch.zeros_like(x)
    cache = s["cache"].double() if "cache" in s else None
    for j in range(longest):
        on = (j < lens).nonzero()[:, 0] if n > 1 else torch.zeros(1, dtype=torch.long, device=x.device)
        at = cu[on] + j
        b = s["B"][at].double().repeat_interleave(rep, 1) * step[at][..., None]
        c = s["C"][at].double().repeat_interleave(rep, 1)
        S[on] = S[on] * keep[at][..., None, None] + b[..., None] * x[at][:, :, None]
        y[at] = torch.einsum("nhk,nhkv->nhv", c, S[on]) + s["D"].double()[:, None] * x[at]
        if cache is not None:
            cache[on, j] = S[on]
    if cache is not None:
        return {"y": y, "cache": cache}
    if s["idx"] is None:
        return {"y": y, "state": S}
    pool = s["state"].double()
    pool[slot] = S
    return {"y": y, "state": pool}


def _exact_verify(s):
    cu, tokens = s["cu"].tolist(), s["tokens"].tolist()
    kept, out = [], []
    for i in range(len(cu) - 1):
        a, b = cu[i], cu[i + 1]
        r = a
        while r < b - 1 and float(s["u"][r]) * float(s["draft"][r, tokens[r + 1]]) < float(s["target"][r, tokens[r + 1]]):
            r += 1
        w = s["target"][r].double()
        if r < b - 1:
            d = (w - s["draft"][r].double()).clamp_min(0.0)
            w = d if bool((d > 0).any()) else w
        kept.append(r - a + 1)
        out.append(int(torch.argmax(w / s["noise"][i].double())))
    return {"kept": torch.tensor(kept, dtype=torch.int32), "token": torch.tensor(out, dtype=torch.int32)}
