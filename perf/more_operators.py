"""A gated linear recurrence with its training, the short convolution's backward pass, and the draw of
tokens from logits, as cases with inputs, a plain form, a 64-bit form and the work that no form can do
without.

  gated_prompt, gated_token  the recurrence h = a h + sqrt(1 - a^2) sigmoid(i) x with a = exp(-exp(A_log)
                             sigmoid(r)), per channel, of packed prompts, and of one token (or a few
                             drafted ones) a request, on a pool of states
  gated_train                its forward and backward pass over packed sequences
  conv_back                  the backward pass of the short causal depthwise convolution
  sample, probs              a token, or the probabilities, from logits under a temperature, top-k, top-p
                             and min-p

``run`` computes a case in elementary torch operations where ``own`` is false, and by the
framework's own calls where it is true.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # The recurrent layer of a hybrid model over the throughput workload's prompts: 32768 tokens as
        # 16 sequences of log-uniform lengths, 32 x 128 channels.
        dict(name="gated prompt 32768x4096", op="gated_prompt", tokens=32768, seqs=16, lens="log", lens_seed=0,
             channels=4096, igate=True, dtype="bf16", pool=True),
        # Many short prompts in fp32, some of them empty, over an odd channel count, without an input gate.
        dict(name="gated prompt ragged fp32", op="gated_prompt", tokens=2741, seqs=37, lens="empty", lens_seed=3,
             channels=1003, igate=False, dtype="fp32", pool=False),
        # A training step's forward and backward pass of that layer, 8 sequences in all.
        dict(name="gated train 16384x4096", op="gated_train", tokens=16384, seqs=8, lens="log", lens_seed=1,
             channels=4096, igate=True, dtype="bf16"),
        # One long document over few channels: only the time axis fills the GPU.
        dict(name="gated train 65536x320", op="gated_train", tokens=65536, seqs=1, lens="log", lens_seed=0,
             channels=320, igate=True, dtype="fp32"),
        # One decode step of 64 requests: a latency-bound call, the smallest.
        dict(name="gated token 64x4096", op="gated_token", rows=64, steps=1, channels=4096, igate=True,
             dtype="bf16", slots=80),
        # Drafted tokens of a large batch: every step's state is kept.
        dict(name="gated draft 512x5", op="gated_token", rows=512, steps=5, channels=2560, igate=True, dtype="bf16",
             slots=530),
        # The backward pass of the convolution of the q, k and v channels (3 x 32 heads x 128).
        dict(name="conv back 32768x12288", op="conv_back", tokens=32768, seqs=16, lens="log", lens_seed=0,
             channels=12288, width=4, silu=True, bias=False, dtype="bf16"),
        # Its odd end: 3 taps, a bias, no activation, fp32, short and empty sequences, no vector access.
        dict(name="conv back ragged fp32", op="conv_back", tokens=2741, seqs=37, lens="empty", lens_seed=3,
             channels=1003, width=3, silu=False, bias=True, dtype="fp32"),
        # A serving batch with a large vocabulary, each request with its own temperature and filters.
        dict(name="sample 64x131072 all", op="sample", rows=64, vocab=131072, filters="all", dtype="fp32"),
        # One request with an odd vocabulary in bf16, where many logits are equal.
        dict(name="sample 1x32003 bf16", op="sample", rows=1, vocab=32003, filters="all", dtype="bf16"),
        # The target's probabilities for the verification of 4 drafted tokens of each of 64 requests.
        dict(name="probs 320x131072 p", op="probs", rows=320, vocab=131072, filters="p", dtype="fp32"),
        # The same for a few rows of a small odd vocabulary.
        dict(name="probs 5x32003 k", op="probs", rows=5, vocab=32003, filters="k", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _channels(rng, hi):
    ch = _log(rng, 16, hi)
    return max(8, ch // 8 * 8) if rng.random() < 0.7 else ch


def draw(rng):
    op = rng.choice(["gated_prompt", "gated_prompt", "gated_train", "gated_train", "gated_token", "conv_back",
                     "conv_back", "sample", "sample", "probs"])
    if op in ("gated_prompt", "gated_train", "conv_back"):
        tokens = _log(rng, 1, 65536)
        case = dict(op=op, tokens=tokens, seqs=min(tokens, _log(rng, 1, 128)), lens=rng.choice(["log", "empty"]),
                    lens_seed=rng.randrange(1 << 20),
                    channels=_channels(rng, min(12288, 2 ** 26 // tokens)))
        case["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        if op == "conv_back":
            return dict(case, width=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7, bias=rng.random() < 0.5)
        case["igate"] = rng.random() < 0.7
        return dict(case, pool=rng.random() < 0.5) if op == "gated_prompt" else case
    if op == "gated_token":
        rows = _log(rng, 1, 1024)
        return dict(op=op, rows=rows, steps=rng.choice([1, 1, 2, 3, 5]), channels=_channels(rng, 8192),
                    igate=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    slots=rows + rng.randrange(1, 40))
    vocab = _log(rng, 500, 200000)
    return dict(op=op, rows=max(1, min(_log(rng, 1, 320), 128 * 131072 // vocab)), vocab=vocab,
                filters=rng.choice(["all", "all", "p", "k", "none"]), dtype=rng.choice(["fp32", "bf16"]))


def lengths(case):
    """Sequence lengths of a case: log-uniform shares of its tokens; "empty": some are 0."""
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

    def slots(rows, count):
        """Distinct slots of the pool; one row of a larger batch is padding (-1: the last slot)."""
        idx = torch.randperm(count - 1, generator=g, device=dev)[:rows].to(torch.int32)
        if rows > 1:
            idx[rows // 2] = -1
        return idx

    op = case["op"]
    st = dict(case=case, op=op)
    if op in ("gated_prompt", "gated_train", "gated_token"):
        dt, ch = DT[case["dtype"]], case["channels"]
        lens = steps_of(case) if op == "gated_token" else lengths(case)
        t, n = sum(lens), len(lens)
        # the gates are slices of one projection; at an open gate a lies between 0.9^8 and 0.999^8
        both = normal(t, 2 * ch).to(dt)
        st.update(cu=_cu(lens, dev), x=normal(t, ch).to(dt), r=both[:, :ch],
                  i=both[:, ch:] if case["igate"] else None,
                  A_log=torch.log(-8.0 * torch.log(0.9 + 0.099 * uniform(ch))))
        if op == "gated_train":
            st.update(state=normal(n, ch), idx=None, dy=normal(t, ch).to(dt), dfinal=normal(n, ch))
        elif op == "gated_prompt" and not case["pool"]:
            st.update(state=normal(n, ch), idx=None)
        else:
            count = case.get("slots", n + 3)
            st.update(state=normal(count, ch), idx=slots(n, count))
        if op == "gated_token" and case["steps"] > 1:
            st.update(cache=torch.zeros(n, case["steps"], ch, device=dev))
    elif op == "conv_back":
        dt, ch, w = DT[case["dtype"]], case["channels"], case["width"]
        lens = lengths(case)
        t, n = sum(lens), len(lens)
        st.update(cu=_cu(lens, dev), x=normal(t, ch).to(dt), dy=normal(t, ch).to(dt),
                  weight=normal(ch, w, std=0.5).to(dt), bias=normal(ch, std=0.1).to(dt) if case["bias"] else None,
                  act="silu" if case["silu"] else None, state=normal(n, w - 1, ch).to(dt),
                  dfinal=normal(n, w - 1, ch).to(dt))
    else:
        n, vocab = case["rows"], case["vocab"]
        st.update(logits=normal(n, vocab, std=2.5).to(DT[case["dtype"]]))
        if op == "sample":
            st.update(noise=torch.empty(n, vocab, device=dev).exponential_(generator=g).clamp_min(1e-30))
        some = case["filters"]
        each = torch.arange(n, device=dev)
        # one request in eight is greedy, as a batch of many users has them; a filter is off for some
        temp = torch.where(each % 8 == 7, 0.0, 0.4 + uniform(n))
        top_k = torch.where(each % 5 == 4, 0, torch.exp(uniform(n) * math.log(1000.0))).to(torch.int32)
        top_p = torch.where(each % 6 == 5, 1.0, 0.7 + 0.29 * uniform(n))
        min_p = torch.where(each % 4 == 3, 0.0, 0.1 * uniform(n))
        st.update(temperature=temp, top_k=top_k if some in ("all", "k") else None,
                  top_p=top_p if some in ("all", "p") else None, min_p=min_p if some == "all" else None)
    return st


# ------------------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import linear_attention_prefill_chunked_gb300 as kda
    op = s["op"]
    if op == "gated_prompt":
        y, final = kda.gated_scan(s["x"], s["r"], s["A_log"], s["cu"], i=s["i"], state=s["state"],
                                  state_indices=s["idx"])
        return {"y": y, "state": final}
    if op == "gated_train":
        y, final, carries = kda.gated_scan(s["x"], s["r"], s["A_log"], s["cu"], i=s["i"], state=s["state"],
                                           output_carries=True)
        dx, dr, di, da_log, dstate = kda.gated_scan_backward(
            s["dy"], s["x"], s["r"], s["A_log"], s["cu"], carries, i=s["i"], state=s["state"], dfinal=s["dfinal"])
        return {"y": y, "state": final, "dx": dx, "dr": dr, "di": di, "dA_log": da_log, "dstate": dstate}
    if op == "gated_token":
        if "cache" in s:
            y = kda.gated_decode_draft(s["x"], s["r"], s["A_log"], s["cu"], s["state"], s["idx"], i=s["i"],
                                       cache=s["cache"], max_steps=s["cache"].shape[1])
            return {"y": y, "cache": s["cache"]}
        y = kda.gated_decode(s["x"], s["r"], s["A_log"], s["state"], s["idx"], i=s["i"])
        return {"y": y, "state": s["state"]}
    if op == "conv_back":
        dx, dw, db, dstate = kda.causal_conv_backward(s["dy"], s["x"], s["weight"], s["cu"], bias=s["bias"],
                                                      activation=s["act"], state=s["state"], dfinal=s["dfinal"])
        return {"dx": dx, "dweight": dw, "dbias": db, "dstate": dstate}
    filters = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    if op == "sample":
        return {"token": kda.sample(s["logits"], s["noise"], **filters)}
    return {"probs": kda.sample_probs(s["logits"], **filters)}


def _run_plain(s):
    op = s["op"]
    if op == "gated_prompt":
        return _plain_prompt(s)[0]
    if op == "gated_train":
        return _plain_train(s)
    if op == "gated_token":
        return _plain_token(s)
    if op == "conv_back":
        return _plain_conv_back(s)
    if op == "sample":
        w = _plain_weights(s)
        score = torch.where(w > 0, w / s["noise"], -1.0)
        best = score.max(1, keepdim=True).values
        vocab = w.shape[1]
        token = torch.where(score == best, torch.arange(vocab, device=w.device), vocab).min(1).values
        return {"token": torch.where(best[:, 0] < 0, -1, token).to(torch.int32)}
    w = _plain_weights(s)
    return {"probs": (w / w.sum(1, keepdim=True)).float()}


def _slot(idx, pool):
    return torch.where(idx < 0, pool.shape[0] - 1, idx).long()


def _places(cu, t):
    """Each token's sequence, its position there, and the sequences' lengths."""
    n = cu.shape[0] - 1
    lens = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(n, device=cu.device), lens, output_size=t)
    return seq, torch.arange(t, device=cu.device) - cu[seq], lens


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, from 0: pairs of steps as one, then the steps between."""
    t = a.shape[0]
    if t == 1:
        return b
    if t % 2:
        a, b = torch.cat([a, a[:1]]), torch.cat([b, b[:1]])
    odd = _scan(a[1::2] * a[::2], a[1::2] * b[::2] + b[1::2])
    before = torch.cat([torch.zeros_like(odd[:1]), odd[:-1]])
    return torch.stack([a[::2] * before + b[::2], odd], 1).flatten(0, 1)[:t]


def _gates(s):
    """sigmoid(r), the log-decay g, the decay a, m = sqrt(1 - a^2), sigmoid(i) and u, in 32 bits."""
    x = s["x"].float()
    sr = torch.sigmoid(s["r"].float())
    g = -torch.exp(s["A_log"]) * sr
    si = torch.ones_like(x) if s["i"] is None else torch.sigmoid(s["i"].float())
    return sr, g, torch.exp(g), torch.sqrt(-torch.expm1(2.0 * g)), si, si * x


def _plain_prompt(s):
    t = s["x"].shape[0]
    cu = s["cu"].long()
    seq, pos, lens = _places(cu, t)
    gates = _gates(s)
    _, _, a, m, _, u = gates
    h0 = s["state"] if s["idx"] is None else s["state"][_slot(s["idx"], s["state"])]
    first = (pos == 0)[:, None]
    h = _scan(torch.where(first, 0.0, a), m * u + torch.where(first, a * h0[seq], 0.0))
    final = torch.where((lens > 0)[:, None], h[(cu[1:] - 1).clamp_min(0)], h0)
    y = h.to(s["x"].dtype)
    if s["idx"] is None:
        return {"y": y, "state": final}, h, gates
    s["state"][_slot(s["idx"], s["state"])] = final
    return {"y": y, "state": s["state"]}, h, gates


def _plain_train(s):
    """The gradients: l_t = dy_t + a_{t+1} l_{t+1}, and from it and the state before each token the rest."""
    out, h, (sr, g, a, m, si, u) = _plain_prompt(s)
    x = s["x"]
    t = x.shape[0]
    cu = s["cu"].long()
    seq, pos, lens = _places(cu, t)
    first, last = (pos == 0)[:, None], (pos == lens[seq] - 1)[:, None]
    before = torch.where(first, s["state"][seq], torch.roll(h, 1, 0))
    after = torch.where(last, 0.0, torch.roll(a, -1, 0))
    grad = s["dy"].float() + torch.where(last, s["dfinal"][seq], 0.0)
    lam = _scan(after.flip(0), grad.flip(0)).flip(0)
    ratio = torch.where(m > 0, g / m, 0.0)
    p = g * a * lam * before - a * a * ratio * u * lam
    dstate = torch.where((lens > 0)[:, None], (a * lam)[cu[:-1].clamp_max(t - 1)], s["dfinal"])
    return dict(out, dx=(m * si * lam).to(x.dtype), dr=(p * (1.0 - sr)).to(x.dtype),
                di=None if s["i"] is None else (m * lam * u * (1.0 - si)).to(x.dtype),
                dA_log=p.double().sum(0).float(), dstate=dstate)


def _plain_token(s):
    x = s["x"]
    t = x.shape[0]
    _, g, a, m, _, u = _gates(s)
    h0 = s["state"][_slot(s["idx"], s["state"])]
    if "cache" not in s:
        h = a * h0 + m * u
        s["state"][_slot(s["idx"], s["state"])] = h
        return {"y": h.to(x.dtype), "state": s["state"]}
    seq, pos, _ = _places(s["cu"].long(), t)
    first = (pos == 0)[:, None]
    h = _scan(torch.where(first, 0.0, a), m * u + torch.where(first, a * h0[seq], 0.0))
    s["cache"][seq, pos] = h
    return {"y": h.to(x.dtype), "cache": s["cache"]}


def _plain_conv_back(s):
    x, w = s["x"], s["weight"].float()
    t, ch = x.shape
    width = w.shape[1]
    cu = s["cu"].long()
    n = cu.shape[0] - 1
    seq, pos, lens = _places(cu, t)
    # each sequence's state, then its tokens: the row that tap j of each token reads
    both = torch.cat([s["state"].reshape(n * (width - 1), ch), x]).float()
    at = pos[:, None] - (width - 1) + torch.arange(width, device=x.device)
    row = torch.where(at >= 0, n * (width - 1) + cu[seq][:, None] + at, (seq * (width - 1))[:, None] + at + width - 1)
    dz = s["dy"].float()
    if s["act"] == "silu":
        z = sum(both[row[:, j]] * w[:, j] for j in range(width))
        z = z if s["bias"] is None else z + s["bias"].float()
        sig = torch.sigmoid(z)
        dz = dz * (sig + z * sig * (1.0 - sig))
    dw = torch.stack([(dz * both[row[:, j]]).sum(0, dtype=torch.float64) for j in range(width)], 1)
    # an input is read by one token at most for each tap
    grad = sum(torch.zeros_like(both).index_copy_(0, row[:, j], dz * w[:, j]) for j in range(width))
    # the last inputs, which are the final state, get its gradient too
    back = (lens[:, None] - (width - 1)) + torch.arange(width - 1, device=x.device)
    each = torch.arange(n, device=x.device)[:, None]
    last = torch.where(back >= 0, n * (width - 1) + cu[:-1, None] + back, each * (width - 1) + back + width - 1)
    grad.index_add_(0, last.flatten(), s["dfinal"].reshape(-1, ch).float())
    return {"dx": grad[n * (width - 1):].to(x.dtype), "dweight": dw.float(),
            "dbias": None if s["bias"] is None else dz.sum(0, dtype=torch.float64).float(),
            "dstate": grad[:n * (width - 1)].view(n, width - 1, ch).to(x.dtype)}


def _plain_weights(s):
    """exp((z - max) / temperature) of the entries that the filters leave, 0 elsewhere; in 64 bits, since an
    entry next to a filter's border stands or falls with the last digits of a sum."""
    z, idx = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    n, vocab = z.shape
    rank = torch.arange(vocab, device=z.device)
    temp = s["temperature"].double()[:, None]
    p = torch.where(temp > 0, torch.exp((z - z[:, :1]) / torch.where(temp > 0, temp, 1.0)), (rank == 0).double())
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        p = torch.where((k <= 0) | (rank < k), p, 0.0)
    if s["top_p"] is not None:
        top_p = s["top_p"].double()[:, None]
        before = torch.cumsum(p, 1) - p
        p = torch.where((rank == 0) | (top_p >= 1.0) | (before < top_p * p.sum(1, keepdim=True)), p, 0.0)
    if s["min_p"] is not None:
        p = torch.where(p >= s["min_p"].double()[:, None], p, 0.0)
    return torch.zeros_like(p).scatter_(1, idx, p)


# ------------------------------------------------------------------------------ the work

def work(case):
    """Bytes of each input read once and each output written once, and the operations of the formulas."""
    size = {"bf16": 2, "fp32": 4}
    op = case["op"]
    if op in ("gated_prompt", "gated_train", "gated_token"):
        e, ch, gates = size[case["dtype"]], case["channels"], 3 + case["igate"]
        lens = steps_of(case) if op == "gated_token" else lengths(case)
        t, n = sum(lens), len(lens)
        row = t * ch * e
        states = 8 * n * ch
        if op == "gated_token":
            if case["steps"] > 1:
                states = 4 * (n + t) * ch
            return {"bytes": gates * row + states + 4 * ch, "flops": 14 * t * ch}
        if op == "gated_prompt":
            return {"bytes": gates * row + states + 4 * ch, "flops": 14 * t * ch}
        return {"bytes": 2 * gates * row + 2 * states + 8 * ch, "flops": 44 * t * ch}
    if op == "conv_back":
        e, ch, w = size[case["dtype"]], case["channels"], case["width"]
        lens = lengths(case)
        t, n = sum(lens), len(lens)
        return {"bytes": 3 * t * ch * e + 3 * n * (w - 1) * ch * e + ch * (w + 1) * (e + 4),
                "flops": t * ch * (6 * w + (8 if case["silu"] else 1))}
    n, vocab = case["rows"], case["vocab"]
    if op == "probs":
        return {"bytes": n * vocab * (size[case["dtype"]] + 4), "flops": 4 * n * vocab}
    # where no filter is on, the noise of every entry is read
    noise = 4 * n * vocab if case["filters"] == "none" else 0
    return {"bytes": n * vocab * size[case["dtype"]] + noise + 4 * n, "flops": 3 * n * vocab}


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions token by token, or row by row, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "conv_back":
        return _exact_conv_back(s)
    if op in ("sample", "probs"):
        return _exact_draw(s)
    return _exact_gated(s)


def _exact_gated(s):
    x, cu = s["x"].double(), s["cu"].long()
    t, ch = x.shape
    n = cu.shape[0] - 1
    lens = cu[1:] - cu[:-1]
    longest = int(lens.max())
    r = s["r"].double()
    rate = torch.exp(s["A_log"].double())
    gate = 1.0 / (1.0 + torch.exp(-r))
    keep = torch.exp(-rate * gate)
    gain = torch.sqrt(-torch.expm1(-2.0 * rate * gate))
    opened = None if s["i"] is None else 1.0 / (1.0 + torch.exp(-s["i"].double()))
    add = gain * (x if opened is None else opened * x)
    slot = torch.arange(n, device=x.device) if s["idx"] is None else _slot(s["idx"], s["state"])
    h = s["state"][slot].double()
    y, held = torch.empty_like(x), torch.empty_like(x)
    cache = s["cache"].double() if "cache" in s else None
    # the sequences by length, longest first: those that still have a token j are the first ones
    order = torch.argsort(lens, descending=True)
    alive = torch.flip(torch.cumsum(torch.flip(torch.bincount(lens, minlength=longest + 1), [0]), 0), [0]).tolist()
    starts, hs = cu[:-1][order], h[order]
    for j in range(longest):
        k = alive[j + 1]
        at = starts[:k] + j
        held[at] = hs[:k]
        hs[:k] = keep[at] * hs[:k] + add[at]
        y[at] = hs[:k]
        if cache is not None:
            cache[order[:k], j] = hs[:k]
    h[order] = hs
    if cache is not None:
        return {"y": y, "cache": cache}
    if s["op"] != "gated_train":
        if s["idx"] is None:
            return {"y": y, "state": h}
        pool = s["state"].double()
        pool[slot] = h
        return {"y": y, "state": pool}
    # what the loss gains from each token's state, last token first
    lam, back = torch.empty_like(x), s["dfinal"].double()[order]
    dy = s["dy"].double()
    for j in range(longest - 1, -1, -1):
        k = alive[j + 1]
        at = starts[:k] + j
        lam[at] = dy[at] + back[:k]
        back[:k] = keep[at] * lam[at]
    dstate = torch.empty_like(back)
    dstate[order] = back
    inner = x if opened is None else opened * x
    d_keep = lam * (held - torch.where(gain > 0, keep / gain, 0.0) * inner)    # by a
    d_gate = d_keep * keep * -rate                                            # by sigmoid(r)
    return {"y": y, "state": h, "dx": lam * gain * (1.0 if opened is None else opened),
            "dr": d_gate * gate * (1.0 - gate),
            "di": None if opened is None else lam * gain * x * opened * (1.0 - opened),
            "dA_log": (d_gate * gate).sum(0), "dstate": dstate}


def _exact_conv_back(s):
    """Sequence by sequence, as gradients of a sum of shifted products."""
    cu = s["cu"].tolist()
    w = s["weight"].double()
    ch, width = w.shape
    dx, dstate = torch.zeros_like(s["x"], dtype=torch.float64), torch.zeros_like(s["state"], dtype=torch.float64)
    dw, db = torch.zeros_like(w), torch.zeros_like(w[:, 0])
    for i in range(len(cu) - 1):
        a, b = cu[i], cu[i + 1]
        ext = torch.cat([s["state"][i], s["x"][a:b]]).double()
        dext = torch.zeros_like(ext)
        dext[b - a:] += s["dfinal"][i].double()
        if b > a:
            z = (ext.unfold(0, width, 1) * w).sum(-1)
            if s["bias"] is not None:
                z = z + s["bias"].double()
            dz = s["dy"][a:b].double()
            if s["act"] == "silu":
                e = torch.exp(-z)
                dz = dz * (1.0 + e + z * e) / (1.0 + e) ** 2
            for j in range(width):
                dext[j:j + b - a] += dz * w[:, j]
                dw[:, j] += (dz * ext[j:j + b - a]).sum(0)
            db += dz.sum(0)
        dstate[i], dx[a:b] = dext[:width - 1], dext[width - 1:]
    return {"dx": dx, "dweight": dw, "dbias": None if s["bias"] is None else db, "dstate": dstate}


def _exact_draw(s):
    tokens, probs = [], torch.zeros(s["logits"].shape, dtype=torch.float64, device=s["logits"].device)
    off = [None] * probs.shape[0]
    temp = s["temperature"].tolist()
    ks, tops, mins = (off if s[k] is None else s[k].tolist() for k in ("top_k", "top_p", "min_p"))
    for i, (t, k, top_p, min_p) in enumerate(zip(temp, ks, tops, mins)):
        z = s["logits"][i].double()
        if t <= 0:
            w = torch.zeros_like(z)
            w[int((z == z.max()).nonzero()[0])] = 1.0
        else:
            order = torch.sort(-z, stable=True).indices
            if k is not None and k > 0:
                order = order[:k]
            w = torch.exp((z[order] - z.max()) / t)
            if top_p is not None and top_p < 1.0:
                sums = torch.cumsum(w, 0)
                order = order[:int((sums < top_p * sums[-1]).sum()) + 1]
            if min_p is not None:
                order = order[w[:order.shape[0]] >= min_p]
            w = torch.zeros_like(z)
            w[order] = torch.exp((z[order] - z.max()) / t)
        probs[i] = w / w.sum()
        if "noise" in s:
            tokens.append(int(torch.argmax(w / s["noise"][i].double())))
    return {"token": torch.tensor(tokens, dtype=torch.int32)} if "noise" in s else {"probs": probs}
